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

// 8 values as they lie in memory: of bf16 only the first 16 bytes are in use.  BF: the
// tensor is known to be bf16 (else `f32` tells, uniformly over the launch), so that the
// second half takes no registers.
template <bool BF> struct Raw { v4u a, b; };
template <> struct Raw<true> { v4u a; };

template <bool BF, bool VEC>
__device__ __forceinline__ void load_raw(const void* p, bool f32, int64_t row_off, int v, int t, int tpr, int d, Raw<BF>& r) {
    const int c = col_of(v, t, tpr);
    r = Raw<BF>{};
    if (VEC ? c < d : c + 8 <= d) {
        if (BF || !f32) {
            r.a = *reinterpret_cast<const typename Aligned<VEC>::bf16*>(static_cast<const uint16_t*>(p) + row_off + c);
        } else if constexpr (!BF) {
            const auto* q = reinterpret_cast<const typename Aligned<VEC>::f32*>(static_cast<const float*>(p) + row_off + c);
            const v4f x = q[0], y = q[1];
            r.a = __builtin_bit_cast(v4u, x);
            r.b = __builtin_bit_cast(v4u, y);
        }
    } else if (!VEC) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (c + j >= d) continue;
            if (BF || !f32) {
                r.a[j / 2] |= (uint32_t)static_cast<const uint16_t*>(p)[row_off + c + j] << (16 * (j % 2));
            } else if constexpr (!BF) {
                const uint32_t w = static_cast<const uint32_t*>(p)[row_off + c + j];
                if (j < 4) r.a[j] = w;
                else r.b[j - 4] = w;
            }
        }
    }
}

template <bool BF>
__device__ __forceinline__ void unpack(const Raw<BF>& r, bool f32, float (&x)[8]) {
    if constexpr (!BF) {
        if (f32) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[j] = __uint_as_float(r.a[j]);
                x[4 + j] = __uint_as_float(r.b[j]);
            }
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = bf16_lo(r.a[j]);
        x[2 * j + 1] = bf16_hi(r.a[j]);
    }
}

// Keeps the compiler from carrying what it unpacked of r before this point past it.
__device__ __forceinline__ void hold(Raw<true>& r) { asm volatile("" : "+v"(r.a)); }
__device__ __forceinline__ void hold(Raw<false>& r) { asm volatile("" : "+v"(r.a), "+v"(r.b)); }

// A row's mean and its sum of squares about the mean, with one barrier: each wave
// finds both of its own values (n of them) in its registers, and the waves' are put
// together by sum(h - m)^2 = sum over the waves of (squares about m_w) + n_w (m_w - m)^2.
template <int NV, bool VEC, bool WAVE_ROW>
__device__ __forceinline__ void mean_and_squares(const float (&h)[NV][8], int t, int tpr, int d, float (*part)[16],
                                                 float& mean, float& squares) {
    auto values_of = [&](int wave) {                  // that the row has in that wave
        int n = 0;
#pragma unroll
        for (int v = 0; v < NV; ++v) n += min(max(d - (v * tpr + wave * 64) * 8, 0), 512);
        return (float)n;
    };
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) s += h[v][j];     // zero past the row's end
    s = wave_sum(s);
    const int wave = __builtin_amdgcn_readfirstlane(WAVE_ROW ? 0 : t >> 6);
    const float n = values_of(wave), m = n == 0.0f ? 0.0f : s / n;
    float q = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = col_of(v, t, tpr);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float e = (VEC ? c < d : c + j < d) ? h[v][j] - m : 0.0f;
            q = __builtin_fmaf(e, e, q);
        }
    }
    q = wave_sum(q);
    if constexpr (WAVE_ROW) {
        mean = m;
        squares = q;
        return;
    }
    if ((t & 63) == 0) {
        part[0][wave] = s;
        part[1][wave] = q;
    }
    // a barrier for LDS alone: loads and stores under way go on
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    const int w = t & 15;                             // 16 lanes hold one wave's each
    const bool in = w < (int)blockDim.x >> 6;
    const float sw = in ? part[0][w] : 0.0f, nw = values_of(w);
    mean = sum16(sw) / (float)d;
    const float off = nw == 0.0f ? 0.0f : sw / nw - mean;
    squares = sum16(in ? __builtin_fmaf(nw * off, off, part[1][w]) : 0.0f);
}

// AHEAD: rows in turn on as many blocks as the card holds, w and b in registers
// throughout, a row's loads sent for before the last one's sums; else a block is one
// row (WAVE_ROW: each of its four waves is one), and only a grid that would pass the
// largest one makes it take more.  10^8 bf16 values with residual, rows in turn / a
// block each, us: rows of 16384 164 / 208, 7168 (16384 rows) 202-210 / 204-247, 5120
// 190 / 194, 8192 164 / 156, 4096 179 / 158, 2048 172 / 164, 1024 180 / 165; of no
// multiple of 8, 2055 287 / 312, 1500 219 / 266, 999 248 / 260, but 333 398 / 361.
// So rows in turn where a row is over 4096 values or not whole vectors, and not a
// wave alone; and not of FP32, whose rows ahead take too many registers.
template <int NV, bool VEC, bool WAVE_ROW, bool BF, bool AHEAD, int MAXT>
__global__ __launch_bounds__(MAXT, NV == 2 ? 4 : 1) void add_layernorm_kernel(AddLayernormArgs a) {
    __shared__ float part[2][2][16];
    const int t = WAVE_ROW ? (int)threadIdx.x & 63 : (int)threadIdx.x;
    const int tpr = WAVE_ROW ? 64 : (int)blockDim.x;
    const int64_t step = WAVE_ROW ? (int64_t)gridDim.x * 4 : gridDim.x;
    const int64_t first = WAVE_ROW ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
    const int d = a.d;
    Raw<BF> x[NV], r[NV];
    auto ask = [&](int64_t row) {
#pragma unroll
        for (int v = 0; v < NV; ++v) load_raw<BF, VEC>(a.x, a.x_f32, row * d, v, t, tpr, d, x[v]);
        if (a.res) {
#pragma unroll
            for (int v = 0; v < NV; ++v) load_raw<BF, VEC>(a.res, a.res_f32, row * d, v, t, tpr, d, r[v]);
        }
    };
    if (AHEAD && first < a.T) ask(first);
    float w[NV][8], b[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        load8<VEC>(a.w, a.w_f32, 0, v, t, tpr, d, w[v]);
        if (a.b) load8<VEC>(a.b, a.w_f32, 0, v, t, tpr, d, b[v]);
    }
    int flip = 0;
    for (int64_t row = first; row < a.T; row += step, flip ^= 1) {
        const int64_t off = row * d;
        if (!AHEAD) ask(row);
        float h[NV][8];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            unpack<BF>(x[v], a.x_f32, h[v]);
            if (a.res) {
                float e[8];
                unpack<BF>(r[v], a.res_f32, e);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[v][j] += e[j];
            }
        }
        if (AHEAD && row + step < a.T) ask(row + step);
        if (a.res && a.h) {
#pragma unroll
            for (int v = 0; v < NV; ++v) store8<VEC, true>(a.h, a.res_f32, off, v, t, tpr, d, h[v]);
        }
        float mean, squares;
        mean_and_squares<NV, VEC, WAVE_ROW>(h, t, tpr, d, part[flip], mean, squares);
        const float rstd = 1.0f / __builtin_sqrtf(squares / (float)d + a.eps);
        if (t == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                y[j] = (h[v][j] - mean) * rstd * w[v][j];
                if (a.b) y[j] += b[v][j];
            }
            if (a.y) store8<VEC, true>(a.y, false, off, v, t, tpr, d, y);
            if constexpr (VEC) {
                if (a.q) store_quant8(a.q, a.scale, row, d, col_of(v, t, tpr), t, y);
            }
        }
    }
}

// Bound by HBM: 8192 rows of 7168 bf16 values with dh 91 to 96 us (4.9 to 5.2 TB/s), and
// 7 for the partial rows.
// AHEAD: a row's dy and h are sent for before the last one's reduction and kept packed.
// IN_LDS: the sums over the rows are kept there, where a row of more than 8192 values
// leaves a thread no registers for them (4096 rows of 16384 bf16 values
// with dh: 116 us, in registers that spill 183 to 250).
template <int NV, bool VEC, bool WAVE_ROW, bool NT, bool BF, bool AHEAD, bool IN_LDS, int MAXT>
__global__ __launch_bounds__(MAXT) void add_layernorm_backward_kernel(AddLayernormBackwardArgs a) {
    __shared__ v4f kept[IN_LDS ? NV * 4 * MAXT : 1];  // [v][dw, db][half of 8][thread]
    auto sums = [&](int v, int which, int half) -> v4f& { return kept[((v * 2 + which) * 2 + half) * MAXT + (int)threadIdx.x]; };
    __shared__ float part[2][2][16];
    const int t = WAVE_ROW ? (int)threadIdx.x & 63 : (int)threadIdx.x;
    const int tpr = WAVE_ROW ? 64 : (int)blockDim.x;
    const int64_t step = WAVE_ROW ? (int64_t)gridDim.x * 4 : gridDim.x;
    const int64_t first = WAVE_ROW ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
    const int d = a.d;
    Raw<BF> next_dy[NV], next_h[NV];
    float next_rstd = 0.0f, next_mean = 0.0f;
    auto ask = [&](int64_t row) {
        if constexpr (AHEAD) {
#pragma unroll
            for (int v = 0; v < NV; ++v) load_raw<BF, VEC>(a.dy, a.dy_f32, row * d, v, t, tpr, d, next_dy[v]);
#pragma unroll
            for (int v = 0; v < NV; ++v) load_raw<BF, VEC>(a.h, a.h_f32, row * d, v, t, tpr, d, next_h[v]);
            next_rstd = a.rstd[row];
            next_mean = a.mean[row];
        }
    };
    if (first < a.T) ask(first);
    float w[NV][8], dw[NV][8], db[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        load8<VEC>(a.w, a.w_f32, 0, v, t, tpr, d, w[v]);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[v][j] = db[v][j] = 0.0f;
        if constexpr (IN_LDS) {
#pragma unroll
            for (int i = 0; i < 4; ++i) sums(v, i >> 1, i & 1) = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        }
    }
    // dw and db of vector v to and from where they are kept (by the thread itself alone)
    auto fetch = [&](int v) {
        if constexpr (IN_LDS) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dw[v][j] = sums(v, 0, j >> 2)[j & 3];
                db[v][j] = sums(v, 1, j >> 2)[j & 3];
            }
        }
    };
    auto keep = [&](int v) {
        if constexpr (IN_LDS) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                sums(v, 0, i) = v4f{dw[v][4 * i], dw[v][4 * i + 1], dw[v][4 * i + 2], dw[v][4 * i + 3]};
                sums(v, 1, i) = v4f{db[v][4 * i], db[v][4 * i + 1], db[v][4 * i + 2], db[v][4 * i + 3]};
            }
        }
    };
    int flip = 0;
    for (int64_t row = first; row < a.T; row += step, flip ^= 1) {
        const int64_t off = row * d;
        float g[NV][8], xh[NV][8], r[AHEAD ? 1 : NV][8];
        Raw<BF> raw_dy[NV], raw_h[NV], raw_dh[NV];
        const float rstd = AHEAD ? next_rstd : a.rstd[row], mean = AHEAD ? next_mean : a.mean[row];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if constexpr (AHEAD) {
                raw_dy[v] = next_dy[v];
                raw_h[v] = next_h[v];
                if (a.dh) load_raw<BF, VEC>(a.dh, a.dx_f32, off, v, t, tpr, d, raw_dh[v]);
            } else {
                load8<VEC>(a.dy, a.dy_f32, off, v, t, tpr, d, g[v]);
                load8<VEC>(a.h, a.h_f32, off, v, t, tpr, d, xh[v]);
                if (a.dh) load8<VEC>(a.dh, a.dx_f32, off, v, t, tpr, d, r[v]);
            }
        }
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if constexpr (AHEAD) {
                unpack<BF>(raw_dy[v], a.dy_f32, g[v]);
                unpack<BF>(raw_h[v], a.h_f32, xh[v]);
            }
            fetch(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {             // past the row's end dy = 0: nothing is added
                xh[v][j] = (xh[v][j] - mean) * rstd;
                dw[v][j] = __builtin_fmaf(g[v][j], xh[v][j], dw[v][j]);
                db[v][j] += g[v][j];
                g[v][j] *= w[v][j];
                s0 += g[v][j];
                s1 = __builtin_fmaf(g[v][j], xh[v][j], s1);
            }
            keep(v);
        }
        if (row + step < a.T) ask(row + step);
        row_sum2<WAVE_ROW>(s0, s1, part[flip]);
        const float c0 = s0 / (float)d, c1 = s1 / (float)d;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if constexpr (AHEAD) {                   // from the packed values again: fewer registers across the sums
                hold(raw_dy[v]);
                hold(raw_h[v]);
                unpack<BF>(raw_dy[v], a.dy_f32, g[v]);
                unpack<BF>(raw_h[v], a.h_f32, xh[v]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    xh[v][j] = (xh[v][j] - mean) * rstd;
                    g[v][j] *= w[v][j];
                }
            }
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = (g[v][j] - c0 - xh[v][j] * c1) * rstd;
            if (a.dh) {
                float e[8];
                if constexpr (AHEAD) unpack<BF>(raw_dh[v], a.dx_f32, e);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] += AHEAD ? e[j] : r[AHEAD ? 0 : v][j];
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
    for (int v = 0; v < NV; ++v) fetch(v);
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

// go<values / 8 of a thread, d % 8 == 0, a row is a wave, most threads>
template <bool FORWARD, typename Launch>
void dispatch_shape(int d, Launch&& go) {
    const bool vec = d % 8 == 0;
    if (d <= 512) {
        vec ? go.template operator()<1, true, true, 256>() : go.template operator()<1, false, true, 256>();
    } else if constexpr (FORWARD) {
        if (d <= 8192) vec ? go.template operator()<2, true, false, 512>() : go.template operator()<2, false, false, 512>();
        else vec ? go.template operator()<2, true, false, 1024>() : go.template operator()<2, false, false, 1024>();
    } else {
        if (d <= 1024) vec ? go.template operator()<2, true, true, 256>() : go.template operator()<2, false, true, 256>();
        else if (d <= 8192) vec ? go.template operator()<1, true, false, 1024>() : go.template operator()<1, false, false, 1024>();
        else vec ? go.template operator()<2, true, false, 1024>() : go.template operator()<2, false, false, 1024>();
    }
}

int forward_threads(int d) { return d <= FORWARD_NARROW ? 256 : (d + 1023) / 1024 * 64; }
int backward_threads(int d) {
    return d <= BACKWARD_NARROW ? 256 : d <= 8192 ? (d + 511) / 512 * 64 : (d + 1023) / 1024 * 64;
}

// As many blocks as the card holds (24 waves of 8 values a thread to a CU, 16 of those
// with sums in LDS), which keeps the partial rows few: 8192 rows of 7168 bf16 values with
// dh on 256 / 512 blocks 110 / 115 us, 16384 of 5120 156 / 136.
int backward_most(int d) {
    const int waves = (d + 511) / 512;
    return d <= 512 ? 1024 : d <= BACKWARD_NARROW ? MOST_PARTIAL_ROWS : d <= 8192 ? 256 * (24 / waves) : 256;
}

// Functions of the sizes alone, so the bits of dw and db are too.
int backward_blocks(int64_t T, int d) {
    const bool narrow = d <= BACKWARD_NARROW;
    const int64_t rows = narrow ? (T + 3) / 4 : T, few = rows / (narrow ? 8 : 4), least = narrow ? 512 : 256;
    const int64_t most = backward_most(d), b = few < least ? least : few < most ? few : most;
    return (int)(rows < b ? rows : b);
}

// Blocks of the forward that goes on from row to row: 16 waves to a CU.
int64_t forward_blocks(int64_t want, int threads) {
    const int64_t most = 256 * (16 / (threads / 64));
    return want < most ? want : most;
}

struct ForwardLaunch {
    const AddLayernormArgs& a;
    hipStream_t st;
    template <int NV, bool VEC, bool WAVE_ROW, int MAXT>
    void operator()() const {
        const int64_t want = WAVE_ROW ? (a.T + 3) / 4 : a.T;
        const int threads = forward_threads(a.d);
        const bool bf = !a.x_f32 && (!a.res || !a.res_f32);
        if (bf && !WAVE_ROW && (!VEC || a.d > 4096))
            hipLaunchKernelGGL((add_layernorm_kernel<NV, VEC, WAVE_ROW, true, true, MAXT>),
                               dim3((unsigned)forward_blocks(want, threads)), dim3(threads), 0, st, a);
        else if (bf)
            hipLaunchKernelGGL((add_layernorm_kernel<NV, VEC, WAVE_ROW, true, false, MAXT>),
                               dim3(launch_blocks(want, threads)), dim3(threads), 0, st, a);
        else
            hipLaunchKernelGGL((add_layernorm_kernel<NV, VEC, WAVE_ROW, false, false, MAXT>),
                               dim3(launch_blocks(want, threads)), dim3(threads), 0, st, a);
    }
};

struct BackwardLaunch {
    const AddLayernormBackwardArgs& a;
    hipStream_t st;
    template <int NV, bool VEC, bool WAVE_ROW, int MAXT>
    void operator()() const {
        const dim3 grid(backward_blocks(a.T, a.d)), block(backward_threads(a.d));
        const bool nt = streamed(a.T * a.d * 2);    // two bytes a value for an FP32 dx too, as the RMS norm's
        constexpr bool WIDE = !WAVE_ROW && NV == 2;
        const bool bf = !a.dy_f32 && !a.h_f32 && !a.dx_f32;
        const auto kernel = bf ? nt ? add_layernorm_backward_kernel<NV, VEC, WAVE_ROW, true, true, true, WIDE, MAXT>
                                    : add_layernorm_backward_kernel<NV, VEC, WAVE_ROW, false, true, true, WIDE, MAXT>
                               : nt ? add_layernorm_backward_kernel<NV, VEC, WAVE_ROW, true, false, !WIDE, WIDE, MAXT>
                                    : add_layernorm_backward_kernel<NV, VEC, WAVE_ROW, false, false, !WIDE, WIDE, MAXT>;
        hipLaunchKernelGGL(kernel, grid, block, 0, st, a);
    }
};

}  // namespace

hipError_t launch_add_layernorm(const AddLayernormArgs& a, hipStream_t st) {
    dispatch_shape<true>(a.d, ForwardLaunch{a, st});
    return hipGetLastError();
}

size_t add_layernorm_backward_ws_bytes(int64_t T, int d) {
    const int64_t most = backward_most(d) < 512 ? 512 : backward_most(d);       // backward_blocks or more
    return 2 * (size_t)(T < most ? T : most) * d * sizeof(float);
}

hipError_t launch_add_layernorm_backward(const AddLayernormBackwardArgs& a, float* dw, float* db, hipStream_t st) {
    int rows = 0;                                   // no rows: the reduction alone, which writes zeros
    if (a.T > 0) {
        dispatch_shape<false>(a.d, BackwardLaunch{a, st});
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        rows = backward_blocks(a.T, a.d);
    }
    hipLaunchKernelGGL(dw_reduce_kernel, dim3((a.d + 15) / 16, db ? 2 : 1), dim3(256), 0, st, a.part, rows, a.d, dw, db);
    return hipGetLastError();
}

}  // namespace moe
