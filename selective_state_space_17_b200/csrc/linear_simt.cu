// linear_simt.cu — matrix product with its epilogue on the general path: fp32
// operands, and 16- or 8-bit operands whose rows TMA cannot address (a pitch or
// a base that is not a multiple of 16 bytes).
//
//     y[m, n] = act(xs[m] ws[n] sum_k x[m, k] w[n, k] + bias[n]) + residual[m, n]
//
// fp32 FMAs on 64 x 64 tiles, 4 x 4 outputs per thread.
#include <algorithm>

#include "layer.cuh"

namespace ssd {
namespace {

constexpr int BM = 64, BN = 64, BK = 16;

template <typename T> __device__ __forceinline__ float load_as_f32(const T* p) { return io<T>::load(p); }
template <> __device__ __forceinline__ float load_as_f32(const __nv_fp8_e4m3* p) { return static_cast<float>(*p); }

template <typename T, typename O>
__global__ void __launch_bounds__(256) linear_simt_kernel(LinearArgs a)
{
    __shared__ float xs[BK][BM + 4], ws[BK][BN + 4];
    const T* x = static_cast<const T*>(a.x);
    const T* w = static_cast<const T*>(a.w);
    const int m0 = blockIdx.x * BM, n0 = blockIdx.y * BN;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += BK) {
#pragma unroll
        for (int i = 0; i < BM * BK / 256; ++i) {
            const int e = threadIdx.x + i * 256, r = e / BK, k = e % BK;
            const bool kin = k0 + k < a.K;
            xs[k][r] = kin && m0 + r < a.M ? load_as_f32(x + (m0 + r) * a.x_stride + k0 + k) : 0.0f;
            ws[k][r] = kin && n0 + r < a.N ? load_as_f32(w + (long long)(n0 + r) * a.K + k0 + k) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < BK; ++k) {
            float xv[4], wv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) { xv[i] = xs[k][ty * 4 + i]; wv[i] = ws[k][tx * 4 + i]; }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xv[i], wv[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + ty * 4 + i;
        if (m >= a.M) break;
        const float sx = a.x_scale ? a.x_scale[m] : 1.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + tx * 4 + j;
            if (n >= a.N) break;
            const long long at = (long long)m * a.N + n;
            float v = acc[i][j];
            if (a.x_scale) v = v * sx * a.w_scale[n];
            if (a.bias) v += a.bias[n];
            v = activate(v, a.act);
            if (a.residual) v += io<O>::load(static_cast<const O*>(a.residual) + at);
            io<O>::store(static_cast<O*>(a.y) + at, v);
        }
    }
}

template <typename T>
cudaError_t launch(const LinearArgs& a, const LaunchCtx& ctx)
{
    const dim3 grid((a.M + BM - 1) / BM, (a.N + BN - 1) / BN);
    if (a.out_bf16) linear_simt_kernel<T, __nv_bfloat16><<<grid, 256, 0, ctx.stream>>>(a);
    else linear_simt_kernel<T, float><<<grid, 256, 0, ctx.stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t linear_simt(const LinearArgs& a, const LaunchCtx& ctx)
{
    switch (a.type) {
    case LinearType::f32: return launch<float>(a, ctx);
    case LinearType::bf16: return launch<__nv_bfloat16>(a, ctx);
    default: return launch<__nv_fp8_e4m3>(a, ctx);
    }
}

}  // namespace ssd
