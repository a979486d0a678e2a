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

// Where a thread's values lie: 8 consecutive ones at column (v tpr + t) 8 - shift for each
// v < NV, t of the row's tpr threads.  In rows of no multiple of 8 the shift is where the
// thread's first row begins in its 16 bytes, and rows 8 apart begin alike, so that the
// accesses stay aligned over its rows; the first and last 8 of a row hold some of the
// neighbouring rows' then, which count as zeros and are not stored.  (60 10^6 values with
// residual, or dh, bf16, before this and several narrow rows to a wave and now, us: 999
// wide 149 -> 111 forward and 205 -> 109 backward, 2055 wide 173 -> 106 and 193 -> 124, 130
// wide 360 -> 163 and 481 -> 163; FP32 67 wide 953 -> 260 and 1126 -> 279; 128 wide, which
// has no shift, 187 -> 80 and 219 -> 90.)
struct Place {
    int t, tpr, shift, d;
    int64_t total;                                    // values of the tensor
    __device__ __forceinline__ int col(int v) const { return (v * tpr + t) * 8 - shift; }
    // values from the row's first to the tensor's end, as far as they matter
    __device__ __forceinline__ int room(int64_t row_off) const {
        const int64_t n = total - row_off;
        return n < 1 << 20 ? (int)n : 1 << 20;
    }
};

// The thread's 8 values of the row at row_off, at vector v.  The tensor's last 8 are read
// where they would go past its end (take_row puts that right).
template <bool BF, bool VEC>
__device__ __forceinline__ void load_raw(const void* p, bool f32, int64_t row_off, int v, const Place& at, Raw<BF>& r) {
    const int c = at.col(v);
    r = Raw<BF>{};
    if (!VEC && at.total < 8) {                       // a tensor of less than 8 values
        uint32_t x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t i = row_off + c + j;
            const bool in = c < at.d && i < at.total;
            x[j] = !in ? 0u : BF || !f32 ? static_cast<const uint16_t*>(p)[i] : static_cast<const uint32_t*>(p)[i];
        }
        if (BF || !f32) r.a = v4u{x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16};
        else if constexpr (!BF) {
            r.a = v4u{x[0], x[1], x[2], x[3]};
            r.b = v4u{x[4], x[5], x[6], x[7]};
        }
    } else if (c < at.d) {
        const int64_t from = row_off + (VEC ? c : min(c, at.room(row_off) - 8));
        if (BF || !f32) {
            r.a = *reinterpret_cast<const typename Aligned<VEC>::bf16*>(static_cast<const uint16_t*>(p) + from);
        } else if constexpr (!BF) {
            const auto* q = reinterpret_cast<const typename Aligned<VEC>::f32*>(static_cast<const float*>(p) + from);
            const v4f x = q[0], y = q[1];
            r.a = __builtin_bit_cast(v4u, x);
            r.b = __builtin_bit_cast(v4u, y);
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

// What load_raw read as the row's own values, zeros in the place of other rows' (unless
// they are not asked for: MASK).
template <bool BF, bool VEC, bool MASK = true>
__device__ __forceinline__ void take_row(const Raw<BF>& r, bool f32, int64_t row_off, int v, const Place& at, float (&x)[8]) {
    unpack<BF>(r, f32, x);
    if constexpr (!VEC) {
        const int c = at.col(v);
        const int room = at.room(row_off);
        if (room < at.d + 8 && at.total >= 8) {       // the last row (of less than 8 values, the last ones)
            const int k = c < at.d ? max(c + 8 - room, 0) : 0;        // values read early
#pragma unroll
            for (int s = 4; s > 0; s >>= 1)
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = !(k & s) ? x[j] : j + s < 8 ? x[j + s] : 0.0f;
        }
        if constexpr (MASK) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = (unsigned)(c + j) < (unsigned)at.d ? x[j] : 0.0f;
        }
    }
}

// 8 values of w or b (zero past the row)
template <bool VEC>
__device__ __forceinline__ void load_weight(const void* p, bool f32, int v, const Place& at, float (&x)[8]) {
    const int c = at.col(v);
    if (VEC ? c < at.d : c >= 0 && c + 8 <= at.d) {
        if (f32) {
            const auto* q = reinterpret_cast<const typename Aligned<VEC>::f32*>(static_cast<const float*>(p) + c);
            const v4f lo = q[0], hi = q[1];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[j] = lo[j];
                x[4 + j] = hi[j];
            }
        } else {
            const v4u q = *reinterpret_cast<const typename Aligned<VEC>::bf16*>(static_cast<const uint16_t*>(p) + c);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[2 * j] = bf16_lo(q[j]);
                x[2 * j + 1] = bf16_hi(q[j]);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = VEC || (unsigned)(c + j) >= (unsigned)at.d ? 0.0f
                   : f32                                     ? static_cast<const float*>(p)[c + j]
                                                             : bf16_to_f32(static_cast<const uint16_t*>(p)[c + j]);
    }
}

template <bool VEC, bool NT>
__device__ __forceinline__ void store_row(void* p, bool f32, int64_t row_off, int v, const Place& at, const float (&x)[8]) {
    const int c = at.col(v);
    if (VEC ? c < at.d : c >= 0 && c + 8 <= at.d) {
        if (f32) {
            typedef typename Aligned<VEC>::f32 V;
            V* q = reinterpret_cast<V*>(static_cast<float*>(p) + row_off + c);
            const V lo = {x[0], x[1], x[2], x[3]}, hi = {x[4], x[5], x[6], x[7]};
            if constexpr (NT) {
                __builtin_nontemporal_store(lo, q);
                __builtin_nontemporal_store(hi, q + 1);
            } else {
                q[0] = lo;
                q[1] = hi;
            }
        } else {
            typedef typename Aligned<VEC>::bf16 V;
            V* q = reinterpret_cast<V*>(static_cast<uint16_t*>(p) + row_off + c);
            const V o = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
            if constexpr (NT) __builtin_nontemporal_store(o, q);
            else *q = o;
        }
    } else if (!VEC) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if ((unsigned)(c + j) >= (unsigned)at.d) continue;
            if (f32) static_cast<float*>(p)[row_off + c + j] = x[j];
            else static_cast<uint16_t*>(p)[row_off + c + j] = (uint16_t)pack_bf16(x[j], 0.0f);
        }
    }
}

// Keeps the compiler from carrying what it unpacked of r before this point past it.
__device__ __forceinline__ void hold(Raw<true>& r) { asm volatile("" : "+v"(r.a)); }
__device__ __forceinline__ void hold(Raw<false>& r) { asm volatile("" : "+v"(r.a), "+v"(r.b)); }

// A row's mean and its sum of squares about the mean, with one barrier: each wave
// finds both of its own values (n of them) in its registers, and the waves' are put
// together by sum(h - m)^2 = sum over the waves of (squares about m_w) + n_w (m_w - m)^2.
// LPR: lanes of a row that a wave has whole, 0 for a block's row.
template <int NV, bool VEC, int LPR>
__device__ __forceinline__ void mean_and_squares(const float (&h)[NV][8], const Place& at, float (*part)[16], float& mean,
                                                 float& squares) {
    const int d = at.d;
    auto values_of = [&](int wave) {                  // that the row has in that wave
        int n = 0;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int from = (v * at.tpr + wave * 64) * 8 - at.shift;
            n += max(min(from + 512, d) - max(from, 0), 0);
        }
        return (float)n;
    };
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) s += h[v][j];     // zero outside the row
    s = lanes_sum<LPR ? LPR : 64>(s);
    const int wave = LPR ? 0 : __builtin_amdgcn_readfirstlane(at.t >> 6);
    const float n = LPR ? (float)d : values_of(wave), m = n == 0.0f ? 0.0f : s / n;
    float q = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = at.col(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float e = (VEC ? c < d : (unsigned)(c + j) < (unsigned)d) ? h[v][j] - m : 0.0f;
            q = __builtin_fmaf(e, e, q);
        }
    }
    q = lanes_sum<LPR ? LPR : 64>(q);
    if constexpr (LPR != 0) {
        mean = m;
        squares = q;
        return;
    }
    if ((at.t & 63) == 0) {
        part[0][wave] = s;
        part[1][wave] = q;
    }
    // a barrier for LDS alone: loads and stores under way go on
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    const int w = at.t & 15;                          // 16 lanes hold one wave's each
    const bool in = w < (int)blockDim.x >> 6;
    const float sw = in ? part[0][w] : 0.0f, nw = values_of(w);
    mean = sum16(sw) / (float)d;
    const float off = nw == 0.0f ? 0.0f : sw / nw - mean;
    squares = sum16(in ? __builtin_fmaf(nw * off, off, part[1][w]) : 0.0f);
}

// The thread's place in its rows, and the first of them and how many on the next is.
template <bool VEC, int LPR>
__device__ __forceinline__ Place place(int64_t T, int d, int64_t& first, int64_t& step) {
    constexpr int PER = LPR ? 256 / LPR : 1;          // rows of a block at a time
    first = LPR ? (int64_t)blockIdx.x * PER + threadIdx.x / (LPR ? LPR : 1) : blockIdx.x;
    step = (int64_t)gridDim.x * PER;
    // the last few widths fill their threads without a shift
    const int shift = VEC || d > 16377 ? 0 : (int)(first * d & 7);
    return Place{LPR ? (int)threadIdx.x % (LPR ? LPR : 1) : (int)threadIdx.x, LPR ? LPR : (int)blockDim.x, shift, d, T * d};
}

// AHEAD: rows in turn on as many blocks as the card holds, w and b in registers
// throughout, a row's loads sent for before the last one's sums; else a block is one
// row (LPR: each LPR lanes are one), and only a grid that would pass the
// largest one makes it take more.  10^8 bf16 values with residual, rows in turn / a
// block each, us: rows of 16384 164 / 208, 7168 (16384 rows) 202-210 / 204-247, 5120
// 190 / 194, 8192 164 / 156, 4096 179 / 158, 2048 172 / 164, 1024 180 / 165; of no
// multiple of 8, 2055 287 / 312, 1500 219 / 266, 999 248 / 260, but 333 398 / 361.
// So rows in turn with the next ones ahead where a row is over 4096 values or not whole
// vectors, and not a wave alone; and not of FP32, whose rows ahead take too many
// registers.  Rows with a shift come in turn in any case, for their weights (FP32, 2055
// wide 169 us, a block each 262; 130 wide 226, 262).
template <int NV, bool VEC, int LPR, bool BF, bool AHEAD, int MAXT>
__global__ __launch_bounds__(MAXT, NV == 2 ? 4 : 1) void add_layernorm_kernel(AddLayernormArgs a) {
    __shared__ float part[2][2][16];
    int64_t first, step;
    const Place at = place<VEC, LPR>(a.T, a.d, first, step);
    const int d = a.d;
    Raw<BF> x[NV], r[NV];
    auto ask = [&](int64_t row) {
#pragma unroll
        for (int v = 0; v < NV; ++v) load_raw<BF, VEC>(a.x, a.x_f32, row * d, v, at, x[v]);
        if (a.res) {
#pragma unroll
            for (int v = 0; v < NV; ++v) load_raw<BF, VEC>(a.res, a.res_f32, row * d, v, at, r[v]);
        }
    };
    if (AHEAD && first < a.T) ask(first);
    float w[NV][8], b[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        load_weight<VEC>(a.w, a.w_f32, v, at, w[v]);
        if (a.b) load_weight<VEC>(a.b, a.w_f32, v, at, b[v]);
    }
    int flip = 0;
    for (int64_t row = first; row < a.T; row += step, flip ^= 1) {
        const int64_t off = row * d;
        if (!AHEAD) ask(row);
        float h[NV][8];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            take_row<BF, VEC>(x[v], a.x_f32, off, v, at, h[v]);
            if (a.res) {
                float e[8];
                take_row<BF, VEC>(r[v], a.res_f32, off, v, at, e);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[v][j] += e[j];
            }
        }
        if (AHEAD && row + step < a.T) ask(row + step);
        if (a.res && a.h) {
#pragma unroll
            for (int v = 0; v < NV; ++v) store_row<VEC, true>(a.h, a.res_f32, off, v, at, h[v]);
        }
        float mean, squares;
        mean_and_squares<NV, VEC, LPR>(h, at, part[flip], mean, squares);
        const float rstd = 1.0f / __builtin_sqrtf(squares / (float)d + a.eps);
        if (at.t == 0) {
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
            if (a.y) store_row<VEC, true>(a.y, false, off, v, at, y);
            if constexpr (VEC) {
                if (a.q) store_quant8(a.q, a.scale, row, d, at.col(v), at.t, y);
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
template <int NV, bool VEC, int LPR, bool NT, bool BF, bool AHEAD, bool IN_LDS, int MAXT>
__global__ __launch_bounds__(MAXT, VEC || IN_LDS ? 1 : LPR || !BF ? 4 : 5) void add_layernorm_backward_kernel(
    AddLayernormBackwardArgs a) {
    __shared__ v4f kept[IN_LDS ? NV * 4 * MAXT : 1];  // [v][dw, db][half of 8][thread]
    auto sums = [&](int v, int which, int half) -> v4f& { return kept[((v * 2 + which) * 2 + half) * MAXT + (int)threadIdx.x]; };
    __shared__ float part[2][2][16];
    int64_t first, step;
    const Place at = place<VEC, LPR>(a.T, a.d, first, step);
    const int d = a.d;
    Raw<BF> next_dy[NV], next_h[NV];
    float next_rstd = 0.0f, next_mean = 0.0f;
    auto ask = [&](int64_t row) {
        if constexpr (AHEAD) {
#pragma unroll
            for (int v = 0; v < NV; ++v) load_raw<BF, VEC>(a.dy, a.dy_f32, row * d, v, at, next_dy[v]);
#pragma unroll
            for (int v = 0; v < NV; ++v) load_raw<BF, VEC>(a.h, a.h_f32, row * d, v, at, next_h[v]);
            next_rstd = a.rstd[row];
            next_mean = a.mean[row];
        }
    };
    if (first < a.T) ask(first);
    float w[NV][8], dw[NV][8], db[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        load_weight<VEC>(a.w, a.w_f32, v, at, w[v]);
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
        float g[NV][8], xh[NV][8];
        Raw<BF> raw_dy[NV], raw_h[NV], raw_dh[NV];
        const float rstd = AHEAD ? next_rstd : a.rstd[row], mean = AHEAD ? next_mean : a.mean[row];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if constexpr (AHEAD) {
                raw_dy[v] = next_dy[v];
                raw_h[v] = next_h[v];
            } else {
                load_raw<BF, VEC>(a.dy, a.dy_f32, off, v, at, raw_dy[v]);
                load_raw<BF, VEC>(a.h, a.h_f32, off, v, at, raw_h[v]);
            }
            if (a.dh) load_raw<BF, VEC>(a.dh, a.dx_f32, off, v, at, raw_dh[v]);
        }
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            take_row<BF, VEC>(raw_dy[v], a.dy_f32, off, v, at, g[v]);
            take_row<BF, VEC>(raw_h[v], a.h_f32, off, v, at, xh[v]);
            fetch(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {             // outside the row dy = 0: nothing is added
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
        if constexpr (LPR != 0) {
            s0 = lanes_sum<LPR>(s0);
            s1 = lanes_sum<LPR>(s1);
        } else {
            row_sum2(s0, s1, part[flip]);
        }
        const float c0 = s0 / (float)d, c1 = s1 / (float)d;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if constexpr (AHEAD) {                   // from the packed values again: fewer registers across the sums
                hold(raw_dy[v]);
                hold(raw_h[v]);
                take_row<BF, VEC, false>(raw_dy[v], a.dy_f32, off, v, at, g[v]);
                take_row<BF, VEC, false>(raw_h[v], a.h_f32, off, v, at, xh[v]);
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
                take_row<BF, VEC, false>(raw_dh[v], a.dx_f32, off, v, at, e);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] += e[j];
            }
            store_row<VEC, NT>(a.dx, a.dx_f32, off, v, at, o);
        }
    }
    if constexpr (LPR != 0) {                            // the block's rows at a time as one partial row, by column
        constexpr int GROUPS = 256 / LPR, WIDE = LPR * 8 * NV;
        __shared__ float sum[GROUPS][WIDE];
        for (int which = 0; which <= (int)a.bias_grad; ++which) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = at.col(v) + j;
                    if ((unsigned)c < (unsigned)d) sum[threadIdx.x / LPR][c] = which ? db[v][j] : dw[v][j];
                }
            __syncthreads();
            for (int c = threadIdx.x; c < d; c += 256) {
                float x[GROUPS];
#pragma unroll
                for (int i = 0; i < GROUPS; ++i) x[i] = sum[i][c];
                a.part[((int64_t)which * gridDim.x + blockIdx.x) * d + c] = pairwise(x);
            }
        }
        return;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) fetch(v);
#pragma unroll
    for (int v = 0; v < NV; ++v) store_row<VEC, false>(a.part, true, (int64_t)blockIdx.x * d, v, at, dw[v]);
    if (a.bias_grad) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            store_row<VEC, false>(a.part, true, ((int64_t)gridDim.x + blockIdx.x) * d, v, at, db[v]);
    }
}

// Values that a row's threads span: of no multiple of 8, up to 7 more.
int span(int d) { return d % 8 == 0 || d > 16377 ? d : d + 7; }
// Lanes of a row that a wave has whole: 8 values (16 in the backward's widest) a lane.
int row_lanes(int d) { return span(d) <= 128 ? 16 : span(d) <= 256 ? 32 : 64; }
constexpr int FORWARD_NARROW = 512;
// Rows of up to 1024 values are a wave's in the backward too, unless they have a shift,
// whose registers leave two such waves to a SIMD (514 wide 189 us, as a block's 182, in
// FP32 310 and 217).
int backward_narrow(int d) { return d % 8 ? 512 : 1024; }

// go<values / 8 of a thread, d % 8 == 0, lanes of a wave's row, most threads>
template <int NV, int LPR, int MAXT, typename Launch>
void go_on(int d, Launch&& go) {
    d % 8 == 0 ? go.template operator()<NV, true, LPR, MAXT>() : go.template operator()<NV, false, LPR, MAXT>();
}
template <bool FORWARD, typename Launch>
void dispatch_shape(int d, Launch&& go) {
    const int n = span(d);
    if (n <= 128) go_on<1, 16, 256>(d, go);
    else if (n <= 256) go_on<1, 32, 256>(d, go);
    else if (n <= 512) go_on<1, 64, 256>(d, go);
    else if constexpr (FORWARD) n <= 8192 ? go_on<2, 0, 512>(d, go) : go_on<2, 0, 1024>(d, go);
    else if (n <= backward_narrow(d)) go.template operator()<2, true, 64, 256>();
    else n <= 8192 ? go_on<1, 0, 1024>(d, go) : go_on<2, 0, 1024>(d, go);
}

int forward_threads(int d) { return span(d) <= FORWARD_NARROW ? 256 : (span(d) + 1023) / 1024 * 64; }
int backward_threads(int d) {
    const int n = span(d);
    return n <= backward_narrow(d) ? 256 : n <= 8192 ? (n + 511) / 512 * 64 : (n + 1023) / 1024 * 64;
}

// As many blocks as the card holds (24 waves of 8 values a thread to a CU, 16 of those
// with a shift or with sums in LDS), which keeps the partial rows few: 8192 rows of 7168
// bf16 values with dh on 256 / 512 blocks 110 / 115 us, 16384 of 5120 156 / 136.
// Narrow rows: 512 wide on 768 / 1024 blocks 89 / 94 us, in FP32 176 / 185; with a shift
// the registers are held to what lets four waves on a SIMD (67 wide on 1024 blocks 176, 768
// 196; in FP32 343 without that, 279 with), and of a block's rows in bf16 five (2055 wide
// 195 -> 124).
int backward_most(int d) {
    const int n = span(d), waves = (n + 511) / 512;
    if (n <= 512) return d % 8 ? 1024 : 768;
    if (n <= backward_narrow(d)) return MOST_PARTIAL_ROWS;
    return n <= 8192 ? 256 * ((d % 8 ? 16 : 24) / waves) : 256;
}

// Functions of the sizes alone, so the bits of dw and db are too.  A multiple of 8 where
// rows come in turn, for the rows' shift.
int backward_blocks(int64_t T, int d) {
    const bool narrow = span(d) <= backward_narrow(d);
    const int per = narrow ? 256 / row_lanes(d) : 1;
    const int64_t rows = (T + per - 1) / per, few = rows / (narrow ? 8 : 4) / 8 * 8, least = narrow ? 512 : 256;
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
    template <int NV, bool VEC, int LPR, int MAXT>
    void operator()() const {
        constexpr int PER = LPR ? 256 / LPR : 1;
        const int64_t want = (a.T + PER - 1) / PER;
        const int threads = forward_threads(a.d);
        const bool bf = !a.x_f32 && (!a.res || !a.res_f32);
        const dim3 turns((unsigned)forward_blocks(want, threads)), grid = VEC ? dim3(launch_blocks(want, threads)) : turns;
        if (bf && !LPR && (!VEC || a.d > 4096))
            hipLaunchKernelGGL((add_layernorm_kernel<NV, VEC, LPR, true, true, MAXT>), turns, dim3(threads), 0, st, a);
        else if (bf)
            hipLaunchKernelGGL((add_layernorm_kernel<NV, VEC, LPR, true, false, MAXT>), grid, dim3(threads), 0, st, a);
        else
            hipLaunchKernelGGL((add_layernorm_kernel<NV, VEC, LPR, false, false, MAXT>), grid, dim3(threads), 0, st, a);
    }
};

struct BackwardLaunch {
    const AddLayernormBackwardArgs& a;
    hipStream_t st;
    template <int NV, bool VEC, int LPR, int MAXT>
    void operator()() const {
        const dim3 grid(backward_blocks(a.T, a.d)), block(backward_threads(a.d));
        const bool nt = streamed(a.T * a.d * 2);    // two bytes a value for an FP32 dx too, as the RMS norm's
        constexpr bool WIDE = !LPR && NV == 2;
        const bool bf = !a.dy_f32 && !a.h_f32 && !a.dx_f32;
        const auto kernel = bf ? nt ? add_layernorm_backward_kernel<NV, VEC, LPR, true, true, true, WIDE, MAXT>
                                    : add_layernorm_backward_kernel<NV, VEC, LPR, false, true, true, WIDE, MAXT>
                               : nt ? add_layernorm_backward_kernel<NV, VEC, LPR, true, false, !WIDE, WIDE, MAXT>
                                    : add_layernorm_backward_kernel<NV, VEC, LPR, false, false, !WIDE, WIDE, MAXT>;
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
