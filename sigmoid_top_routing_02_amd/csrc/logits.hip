// The router's backward from a gradient of all its logits, FP32 [T, E]:
//     du = du_in + dlogits . e    (e = centroids, bf16 [E, d]),
//     de = de_in + dlogits^T . u  (u bf16 [T, d]).
// moe_router_backward takes the gates' gradient, K values a token; what the balance
// loss adds is dense.
#include "device_math.h"
#include "kernels.h"

namespace moe {
namespace {

// C[M, N] = in + A B, A FP32 (A_T: stored [K, M], else [M, K]), B bf16 [K, N], N % 64
// == 0: tiles of 64 x 64, 16 of K at a time, 4 x 4 outputs a thread.
template <bool A_T>
__global__ __launch_bounds__(256) void logits_gemm_kernel(const float* __restrict__ a, const uint16_t* __restrict__ b,
                                                          int64_t M, int N, int64_t K, const float* in, float* out) {
    __shared__ float as[16][65], bs[16][64];
    const int tid = threadIdx.x, n0 = blockIdx.x * 64;
    const int64_t m0 = (int64_t)blockIdx.y * 64;
    const int tm = (tid >> 4) * 4, tn = (tid & 15) * 4;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < K; k0 += 16) {
        for (int i = tid; i < 1024; i += 256) {
            const int m = A_T ? i & 63 : i >> 4, k = A_T ? i >> 6 : i & 15;
            const bool in_a = m0 + m < M && k0 + k < K;
            as[k][m] = in_a ? a[A_T ? (k0 + k) * M + m0 + m : (m0 + m) * K + k0 + k] : 0.0f;
            bs[i >> 6][i & 63] = k0 + (i >> 6) < K ? bf16_to_f32(b[(k0 + (i >> 6)) * N + n0 + (i & 63)]) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_fmaf(as[k][tm + i], bs[k][tn + j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i) {
        if (m0 + tm + i >= M) break;
        for (int j = 0; j < 4; ++j) {
            const int64_t at = (m0 + tm + i) * N + n0 + tn + j;
            out[at] = (in ? in[at] : 0.0f) + acc[i][j];
        }
    }
}

}  // namespace

size_t router_logits_backward_ws_bytes(int64_t T, int d, int E) { return 16; }

hipError_t launch_router_logits_backward(const float* dlogits, const uint16_t* u, const uint16_t* e, int64_t T, int d,
                                         int E, const float* du_in, const float* de_in, float* du, float* de, void* ws,
                                         hipStream_t st) {
    if (du && T > 0)
        hipLaunchKernelGGL((logits_gemm_kernel<false>), dim3(d / 64, (unsigned)((T + 63) / 64)), dim3(256), 0, st, dlogits,
                           e, T, d, (int64_t)E, du_in, du);
    if (de)
        hipLaunchKernelGGL((logits_gemm_kernel<true>), dim3(d / 64, (E + 63) / 64), dim3(256), 0, st, dlogits, u,
                           (int64_t)E, d, T, de_in, de);
    return hipGetLastError();
}

}  // namespace moe
