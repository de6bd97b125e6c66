// linear_simt.cu — matrix product with its epilogue beside the tensor cores:
//
//     y[m, n] = act(xs[m] ws[n] sum_k x[m, k] w[n, k] + bias[n]) + residual[m, n]
//
// linear_rows: few tokens whose operands the tensor-core kernels cannot take as
// they lie (fp32, or rows that TMA cannot address); linear_simt: any operands,
// the kernel of last resort; and the packing of such operands for the
// tensor-core kernels when there are more tokens. Measured: one token, 2560 x 5120 in
// fp32 20 us and 10576 x 2561 in bf16 24 us with the host's share; 17 tokens of 2560 x
// 2561 in bf16, copy included, 24 us.
#include <algorithm>

#include "layer.cuh"

namespace ssd {
namespace {

constexpr int BM = 64, BN = 64, BK = 16;

template <typename T> __device__ __forceinline__ float load_as_f32(const T* p) { return io<T>::load(p); }
template <> __device__ __forceinline__ float load_as_f32(const __nv_fp8_e4m3* p) { return static_cast<float>(*p); }

template <typename O>
__device__ __forceinline__ void finish(const LinearArgs& a, int m, int n, float v)
{
    const long long at = (long long)m * a.N + n;
    if (a.x_scale) v = v * a.x_scale[m] * a.w_scale[n];
    if (a.bias) v += a.bias[n];
    v = activate<O>(v, a.act);
    // residual may be y itself: a plain load
    if (a.residual) v += static_cast<float>(static_cast<const O*>(a.residual)[at]);
    io<O>::store(static_cast<O*>(a.y) + at, v);
}

// fp32 FMAs on 64 x 64 tiles, 4 x 4 outputs per thread. With `only_if`, runs
// only when that word is not zero (see linear_split in linear.cu).
template <typename T, typename O>
__global__ void __launch_bounds__(256) linear_simt_kernel(LinearArgs a, const unsigned int* only_if)
{
    __shared__ float xs[BK][BM + 4], ws[BK][BN + 4];
    if (only_if && *only_if == 0) return;
    const T* x = static_cast<const T*>(a.x);
    const T* w = static_cast<const T*>(a.w);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int tn = (a.N + BN - 1) / BN;
    const long long tiles = (long long)((a.M + BM - 1) / BM) * tn;
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int m0 = (int)(tile / tn) * BM, n0 = (int)(tile % tn) * BN;
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
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + tx * 4 + j;
                if (n < a.N) finish<O>(a, m, n, acc[i][j]);
            }
        }
    }
}

// MT tokens x CH channels per CTA: its warps take every eighth piece of 32 * VEC
// of the K axis, so the weights are read once, in whole lines, and a call with
// few channels still has many loads in flight; the lanes' and the warps' parts
// are added up in a fixed order. Bound by the weights' bytes.
constexpr int kRowWarps = 8;

template <typename T, typename O, int MT, int CH, int VEC>
__global__ void __launch_bounds__(32 * kRowWarps) linear_rows_kernel(LinearArgs a)
{
    __shared__ float part[kRowWarps][MT * CH];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n0 = blockIdx.x * CH, m0 = blockIdx.y * MT;
    const T* x = static_cast<const T*>(a.x);
    const T* w = static_cast<const T*>(a.w);
    float acc[MT][CH] = {};
#pragma unroll(MT > 4 ? 2 : 4)
    for (int k = (warp * 32 + lane) * VEC; k < a.K; k += 32 * kRowWarps * VEC) {
        float wv[CH][VEC];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const T* p = w + (long long)min(n0 + c, a.N - 1) * a.K + k;
            if constexpr (VEC > 1) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(p));
                wv[c][0] = f.x; wv[c][1] = f.y; wv[c][2] = f.z; wv[c][3] = f.w;
            } else {
                wv[c][0] = load_as_f32(p);
            }
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            float xv[VEC];
            const T* p = x + (long long)min(m0 + i, a.M - 1) * a.x_stride + k;
            if constexpr (VEC > 1) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(p));
                xv[0] = f.x; xv[1] = f.y; xv[2] = f.z; xv[3] = f.w;
            } else {
                xv[0] = load_as_f32(p);
            }
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int j = 0; j < VEC; ++j) acc[i][c] = fmaf(xv[j], wv[c][j], acc[i][c]);
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int c = 0; c < CH; ++c) {
#pragma unroll
            for (int o = 16; o; o >>= 1) acc[i][c] += __shfl_xor_sync(0xffffffffu, acc[i][c], o);
            if (lane == 0) part[warp][i * CH + c] = acc[i][c];
        }
    __syncthreads();
    if (threadIdx.x < MT * CH) {
        const int m = m0 + threadIdx.x / CH, n = n0 + threadIdx.x % CH;
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < kRowWarps; ++k) v += part[k][threadIdx.x];
        if (m < a.M && n < a.N) finish<O>(a, m, n, v);
    }
}

template <typename T, typename O, int VEC>
cudaError_t launch_rows(const LinearArgs& a, const LaunchCtx& ctx)
{
    const auto grid = [&](int mt, int ch) { return dim3((a.N + ch - 1) / ch, (a.M + mt - 1) / mt); };
    if (a.M == 1) linear_rows_kernel<T, O, 1, 4, VEC><<<grid(1, 4), 32 * kRowWarps, 0, ctx.stream>>>(a);
    else if (a.M <= 4) linear_rows_kernel<T, O, 4, 4, VEC><<<grid(4, 4), 32 * kRowWarps, 0, ctx.stream>>>(a);
    else linear_rows_kernel<T, O, 8, 8, VEC><<<grid(8, 8), 32 * kRowWarps, 0, ctx.stream>>>(a);
    return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t rows_out(const LinearArgs& a, const LaunchCtx& ctx)
{
    return a.out_bf16 ? launch_rows<T, __nv_bfloat16, VEC>(a, ctx) : launch_rows<T, float, VEC>(a, ctx);
}

template <typename T>
cudaError_t launch_simt(const LinearArgs& a, const unsigned int* only_if, const LaunchCtx& ctx)
{
    const long long tiles = (long long)((a.N + BN - 1) / BN) * ((a.M + BM - 1) / BM);
    const unsigned grid = (unsigned)std::min<long long>(tiles, 2ll * ctx.num_sms);
    if (a.out_bf16) linear_simt_kernel<T, __nv_bfloat16><<<grid, 256, 0, ctx.stream>>>(a, only_if);
    else linear_simt_kernel<T, float><<<grid, 256, 0, ctx.stream>>>(a, only_if);
    return cudaGetLastError();
}

// A CTA to 1024 elements of a row, four to a thread, a CTA's width apart.
constexpr int kPackThreads = 256, kPackEach = 4;

template <typename T>
__global__ void __launch_bounds__(kPackThreads) pack_rows_kernel(const T* src, long long stride, int K, T* dst, int pitch)
{
    const T* s = src + blockIdx.x * stride;
    T* d = dst + (long long)blockIdx.x * pitch;
    const int k0 = blockIdx.y * kPackThreads * kPackEach + threadIdx.x;
    T v[kPackEach];
#pragma unroll
    for (int i = 0; i < kPackEach; ++i) {
        const int k = k0 + i * kPackThreads;
        v[i] = k < K ? s[k] : T(0);
    }
#pragma unroll
    for (int i = 0; i < kPackEach; ++i) {
        const int k = k0 + i * kPackThreads;
        if (k < pitch) d[k] = v[i];
    }
}

// fp32 as the sum of three bf16, 24 significant bits in all: each is what the
// ones before it leave, rounded, and the differences are exact. Where the parts are
// not the value the flag is set: infinities, NaN, values that round to infinity, and
// those below 2^-109 whose last bits lie below bf16's smallest value, 2^-133.
__global__ void __launch_bounds__(kPackThreads) split_rows_kernel(const float* src, long long stride, int K,
                                                                  __nv_bfloat16* dst, int section, unsigned int* flag)
{
    const float* s = src + blockIdx.x * stride;
    __nv_bfloat16* d = dst + (long long)blockIdx.x * 3 * section;
    const int k0 = blockIdx.y * kPackThreads * kPackEach + threadIdx.x;
    float v[kPackEach];
    bool odd = false;
#pragma unroll
    for (int i = 0; i < kPackEach; ++i) {
        const int k = k0 + i * kPackThreads;
        v[i] = k < K ? s[k] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kPackEach; ++i) {
        const int k = k0 + i * kPackThreads;
        if (k >= section) break;
        const __nv_bfloat16 b1 = __float2bfloat16_rn(v[i]);
        const float r1 = v[i] - __bfloat162float(b1);
        const __nv_bfloat16 b2 = __float2bfloat16_rn(r1);
        const float r2 = r1 - __bfloat162float(b2);
        const __nv_bfloat16 b3 = __float2bfloat16_rn(r2);
        d[k] = b1;
        d[section + k] = b2;
        d[2 * section + k] = b3;
        odd |= !(__bfloat162float(b3) == r2);  // also where r2 is NaN: inf - inf
    }
    if (odd) *flag = 1u;  // every writer writes the same
}

dim3 pack_grid(int rows, int pitch)
{
    return dim3(rows, (pitch + kPackThreads * kPackEach - 1) / (kPackThreads * kPackEach));
}

}  // namespace

cudaError_t linear_simt(const LinearArgs& a, const unsigned int* only_if, const LaunchCtx& ctx)
{
    switch (a.type) {
    case LinearType::f32: return launch_simt<float>(a, only_if, ctx);
    case LinearType::bf16: return launch_simt<__nv_bfloat16>(a, only_if, ctx);
    default: return launch_simt<__nv_fp8_e4m3>(a, only_if, ctx);
    }
}

cudaError_t linear_rows(const LinearArgs& a, const LaunchCtx& ctx)
{
    switch (a.type) {
    case LinearType::f32:
        if (a.K % 4 == 0 && a.x_stride % 4 == 0 && aligned_to(a.x, 16)) return rows_out<float, 4>(a, ctx);
        return rows_out<float, 1>(a, ctx);
    case LinearType::bf16: return rows_out<__nv_bfloat16, 1>(a, ctx);
    default: return rows_out<__nv_fp8_e4m3, 1>(a, ctx);
    }
}

cudaError_t pack_rows(const void* src, long long stride, int rows, int K, LinearType type, void* dst, int pitch,
                      const LaunchCtx& ctx)
{
    const dim3 grid = pack_grid(rows, pitch);
    if (type == LinearType::bf16)
        pack_rows_kernel<<<grid, kPackThreads, 0, ctx.stream>>>(static_cast<const uint16_t*>(src), stride, K,
                                                       static_cast<uint16_t*>(dst), pitch);
    else
        pack_rows_kernel<<<grid, kPackThreads, 0, ctx.stream>>>(static_cast<const uint8_t*>(src), stride, K,
                                                       static_cast<uint8_t*>(dst), pitch);
    return cudaGetLastError();
}

cudaError_t split_rows(const float* src, long long stride, int rows, int K, void* dst, int section,
                       unsigned int* flag, const LaunchCtx& ctx)
{
    split_rows_kernel<<<pack_grid(rows, section), kPackThreads, 0, ctx.stream>>>(
        src, stride, K, static_cast<__nv_bfloat16*>(dst), section, flag);
    return cudaGetLastError();
}

}  // namespace ssd
