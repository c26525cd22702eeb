// The router projection's gradient from that of its logits:
//   dx[t, n] = dx_in[t, n] + sum_e dl[t, e] w[e, n],   dw[e, n] = sum_t dl[t, e] x[t, n]
// in fp32.  64x64 tiles, 16 of the reduction per stage through LDS, 4x4 sums per
// thread.
#include "device.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kE = 256;
constexpr int kT = 64, kK = 16;

// C[m, n] = C_in[m, n] + sum_k A(m, k) B(k, n); A(m, k) = a[m*256 + k] (M = T, K =
// 256) or, transposed, a[k*256 + m] (M = 256, K = T); B(k, n) = b[k*N + n].
template <bool TRANS, bool B16>
__global__ __launch_bounds__(256) void k_tile_gemm(int M, int N, int K, const float *__restrict__ a,
                                                   const void *__restrict__ b, const float *__restrict__ cin,
                                                   float *__restrict__ c) {
    __shared__ float sa[kK][kT + 4], sb[kK][kT + 4];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int64_t m0 = (int64_t)blockIdx.y * kT;
    const int n0 = blockIdx.x * kT;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < K; k0 += kK) {
        __syncthreads();
        for (int i = tid; i < kK * kT; i += 256) {
            const int k = TRANS ? i / kT : i % kK, m = TRANS ? i % kT : i / kK;
            const bool in = m0 + m < M && k0 + k < K;
            sa[k][m] = !in ? 0.f : TRANS ? a[(int64_t)(k0 + k) * kE + m0 + m] : a[(m0 + m) * kE + k0 + k];
            const int kb = i / kT, n = i % kT;
            const int64_t at = (int64_t)(k0 + kb) * N + n0 + n;
            sb[kb][n] = k0 + kb >= K ? 0.f
                        : B16        ? bf16_to_f32(static_cast<const uint16_t *>(b)[at])
                                     : static_cast<const float *>(b)[at];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kK; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += sa[k][ty * 4 + i] * sb[k][tx * 4 + j];
    }
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty * 4 + i;
        if (m >= M) continue;
        for (int j = 0; j < 4; ++j) {
            const int64_t at = m * N + n0 + tx * 4 + j;
            c[at] = acc[i][j] + (cin ? cin[at] : 0.f);
        }
    }
}

}  // namespace

size_t router_grad_ws_bytes(int, int, bool) { return 0; }

hipError_t launch_router_grad(const RouterGradArgs &a, void *, hipStream_t s) {
    const dim3 block(256), gx(a.d / kT, (a.T + kT - 1) / kT), gw(a.d / kT, kE / kT);
    hipLaunchKernelGGL((k_tile_gemm<false, false>), gx, block, 0, s, a.T, a.d, kE, a.dlogits, a.w, a.dx_in, a.dx);
    if (a.x_bf16)
        hipLaunchKernelGGL((k_tile_gemm<true, true>), gw, block, 0, s, kE, a.d, a.T, a.dlogits, a.x, nullptr, a.dw);
    else
        hipLaunchKernelGGL((k_tile_gemm<true, false>), gw, block, 0, s, kE, a.d, a.T, a.dlogits, a.x, nullptr, a.dw);
    return hipGetLastError();
}

}  // namespace moe
