// norm.cu — root-mean-square norm with the residual's addition or the gate,
// and an output in the I/O dtype or in 8 bits with one scale per row.
//
//     v = x + r  (r_out = v)   or   v = x silu(z)   or   v = x
//     y_j = v_j w_j rho_g,  rho_g = 1 / sqrt(mean over group g of v^2 + eps)
//     8 bits: s = max(max_j |y_j| / 448, 2^-126),  q_j = e4m3(y_j / s)
//
// Bound by HBM: every element is read and written once, about ten operations
// each. The row stays in registers between the reduction and the output, and
// one reduction serves both: rho_g is constant over a group, so max |y| is the
// maximum over the groups of rho_g max |v w| and needs no second pass.
#include <algorithm>

#include "layer.cuh"

namespace ssd {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kScaleMin = 1.17549435e-38f;  // 2^-126

enum Mode { kPlain = 0, kResidual = 1, kGate = 2 };

// Larger of two values, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float2 warp_sum_max(float2 v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y = max_nan(v.y, __shfl_xor_sync(0xffffffffu, v.y, o));
    }
    return v;
}

template <int VEC>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float* v)
{
    if constexpr (VEC == 1) {
        *p = __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
    } else {
        uint32_t w[VEC / 4];
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]),
                                                         __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]),
                                                         __NV_SATFINITE, __NV_E4M3);
            w[i] = lo | (hi << 16);
        }
        if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
        else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
}

// A row is spread over `groups` x `wpg` warps, whole warps to one group, and
// each lane takes vectors of VEC elements, wpg * 32 vectors apart. With VPT > 0
// a lane has at most VPT of them and keeps them in registers; VPT = 0 takes any
// width and reads the row a second time for the output. When a row fits one
// warp a CTA runs blockDim / 32 rows at a time and needs no barrier.
template <typename T, typename R, int MODE, bool Q8, int VEC, int VPT>
__global__ void __launch_bounds__(1024)
rms_norm_kernel(NormArgs a, int wpg)
{
    __shared__ float2 red[2][32];
    constexpr bool kKeep = VPT > 0;
    constexpr int kV = kKeep ? VPT : 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int wpr = a.groups * wpg;               // warps of a row
    const int rows_per_cta = wpr == 1 ? (int)(blockDim.x >> 5) : 1;
    const int wr = wpr == 1 ? 0 : warp;           // this warp within its row
    const int group = wr / wpg;
    const int Dg = a.D / a.groups;
    const int nvec = Dg / VEC;                    // vectors of a group
    const int t0 = (wr - group * wpg) * 32 + lane, stride = wpg * 32;
    const long long gbase = (long long)group * Dg;
    const T* x = static_cast<const T*>(a.x);
    const R* res = static_cast<const R*>(a.residual);
    const T* gate = static_cast<const T*>(a.gate);
    R* res_out = static_cast<R*>(a.residual_out);
    int buf = 0;

    // sum of squares and max |v w| of one vector; v into val, v w into vw
    auto combine = [&](const Packed<T, VEC>& px, const Packed<T, VEC>& pz, const Packed<R, VEC>& pr,
                       float* val) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            float v = px.get(j);
            if constexpr (MODE == kResidual) v += pr.get(j);
            if constexpr (MODE == kGate) v *= silu_f(pz.get(j));
            val[j] = v;
        }
    };

    for (long long row = (long long)blockIdx.x * rows_per_cta + (wpr == 1 ? warp : 0); row < a.rows;
         row += (long long)gridDim.x * rows_per_cta) {
        const long long base = row * a.D + gbase;
        const long long zbase = row * a.gate_stride + gbase;
        float val[kV][VEC];
        float2 acc = make_float2(0.0f, 0.0f);
        const int iters = kKeep ? kV : (nvec + stride - 1 - t0) / stride;
        auto load_combine = [&](int i, float* v) {
            const long long c = (long long)(t0 + i * stride) * VEC;
            Packed<T, VEC> px, pz;
            Packed<R, VEC> pr;
            px.load(x + base + c);
            if constexpr (MODE == kGate) pz.load(gate + zbase + c);
            if constexpr (MODE == kResidual) pr.load(res + base + c);
            combine(px, pz, pr, v);
        };
        if constexpr (kKeep) {
            Packed<T, VEC> px[kV], pz[kV];
            Packed<R, VEC> pr[kV];
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                px[i].zero(); pz[i].zero(); pr[i].zero();
                if (t0 + i * stride < nvec) {
                    const long long c = (long long)(t0 + i * stride) * VEC;
                    px[i].load(x + base + c);
                    if constexpr (MODE == kGate) pz[i].load(gate + zbase + c);
                    if constexpr (MODE == kResidual) pr[i].load(res + base + c);
                }
            }
#pragma unroll
            for (int i = 0; i < kV; ++i) combine(px[i], pz[i], pr[i], val[i]);
        }
#pragma unroll
        for (int i = 0; i < iters; ++i) {
            if (t0 + i * stride >= nvec) break;
            float* v = val[kKeep ? i : 0];
            if constexpr (!kKeep) load_combine(i, v);
            float wv[VEC];
            if constexpr (Q8) {
                Packed<float, VEC> pw;
                pw.load(a.weight + gbase + (long long)(t0 + i * stride) * VEC);
#pragma unroll
                for (int j = 0; j < VEC; ++j) wv[j] = pw.get(j);
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                acc.x = fmaf(v[j], v[j], acc.x);
                if constexpr (Q8) acc.y = max_nan(acc.y, fabsf(v[j] * wv[j]));
            }
        }
        acc = warp_sum_max(acc);
        float amax_y = 0.0f;
        if (wpr > 1) {
            // two buffers: a warp writes the next row's only after this row's
            // barrier, which follows every read of the buffer before it
            if (lane == 0) red[buf][warp] = acc;
            __syncthreads();
            float sum = 0.0f;
            if (a.groups == 1) {
                acc = warp_sum_max(lane < wpr ? red[buf][lane] : make_float2(0.0f, 0.0f));
                sum = acc.x;
                if constexpr (Q8) amax_y = acc.y * rsqrtf(sum / (float)Dg + a.eps);
            } else {
                for (int g = 0; g < a.groups; ++g) {
                    float2 t = make_float2(0.0f, 0.0f);
                    for (int k = 0; k < wpg; ++k) {
                        const float2 e = red[buf][g * wpg + k];
                        t.x += e.x;
                        t.y = max_nan(t.y, e.y);
                    }
                    if (g == group) sum = t.x;
                    if constexpr (Q8) amax_y = max_nan(amax_y, t.y * rsqrtf(t.x / (float)Dg + a.eps));
                }
            }
            acc.x = sum;
            buf ^= 1;
        } else if constexpr (Q8) {
            amax_y = acc.y * rsqrtf(acc.x / (float)Dg + a.eps);
        }
        const float rho = rsqrtf(acc.x / (float)Dg + a.eps);
        float inv = 1.0f;
        if constexpr (Q8) {
            const float s = max_nan(amax_y / kE4m3Max, kScaleMin);
            if (wr == 0 && lane == 0) a.scale[row] = s;
            inv = 1.0f / s;
        }
#pragma unroll
        for (int i = 0; i < iters; ++i) {
            if (t0 + i * stride >= nvec) break;
            const long long c = (long long)(t0 + i * stride) * VEC;
            float* v = val[kKeep ? i : 0];
            if constexpr (!kKeep) load_combine(i, v);
            if constexpr (MODE == kResidual) {
                if (res_out) {
                    Packed<R, VEC> po;
                    po.set(v);
                    po.store(res_out + base + c);
                }
            }
            Packed<float, VEC> pw;
            pw.load(a.weight + gbase + c);
            float o[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                o[j] = v[j] * pw.get(j) * rho;
                if constexpr (Q8) o[j] *= inv;
            }
            if constexpr (Q8) {
                store_e4m3<VEC>(static_cast<uint8_t*>(a.y) + base + c, o);
            } else {
                Packed<T, VEC> po;
                po.set(o);
                po.store(static_cast<T*>(a.y) + base + c);
            }
        }
    }
}

template <typename T, typename R, int MODE, bool Q8, int VEC, int VPT>
cudaError_t launch(const NormArgs& a, const LaunchCtx& ctx)
{
    const int nvec = a.D / a.groups / VEC;
    const int most = 32 / a.groups;  // warps a group may have
    int wpg = VPT ? (nvec + 32 * VPT - 1) / (32 * VPT) : std::min(most, (nvec + 31) / 32);
    wpg = std::max(1, std::min(wpg, most));
    const int wpr = wpg * a.groups;
    const int threads = wpr == 1 ? 128 : wpr * 32;
    const long long ctas = wpr == 1 ? (a.rows + 3) / 4 : a.rows;
    const long long cap = (long long)ctx.num_sms * std::max(1, 2048 / threads);
    rms_norm_kernel<T, R, MODE, Q8, VEC, VPT>
        <<<(unsigned)std::min(ctas, cap), threads, 0, ctx.stream>>>(a, wpg);
    return cudaGetLastError();
}

// The widest access that every row allows (16 bytes of the I/O dtype), and the
// fewest vectors per lane that put a group in registers.
template <typename T, typename R, int MODE, bool Q8>
cudaError_t pick(const NormArgs& a, const LaunchCtx& ctx)
{
    constexpr int V = 16 / (int)sizeof(T);
    const int Dg = a.D / a.groups;
    const bool vec = Dg % V == 0 &&
                     (MODE != kGate || (aligned_to(a.gate, 16) && a.gate_stride % V == 0));
    const int lanes = 32 * (32 / a.groups);  // lanes a group may have in a CTA of 1024
    const int n = vec ? Dg / V : Dg;
    if (vec) {
        if (n <= lanes) return launch<T, R, MODE, Q8, V, 1>(a, ctx);
        if (n <= 2 * lanes) return launch<T, R, MODE, Q8, V, 2>(a, ctx);
        return launch<T, R, MODE, Q8, V, 0>(a, ctx);
    }
    if (n <= 4 * lanes) return launch<T, R, MODE, Q8, 1, 4>(a, ctx);
    return launch<T, R, MODE, Q8, 1, 0>(a, ctx);
}

template <typename T, typename R, int MODE>
cudaError_t pick_out(const NormArgs& a, const LaunchCtx& ctx)
{
    return a.scale ? pick<T, R, MODE, true>(a, ctx) : pick<T, R, MODE, false>(a, ctx);
}

template <typename T>
cudaError_t pick_mode(const NormArgs& a, const LaunchCtx& ctx)
{
    if (a.gate) return pick_out<T, T, kGate>(a, ctx);
    if (!a.residual) return pick_out<T, T, kPlain>(a, ctx);
    if (a.res_f32) return pick_out<T, float, kResidual>(a, ctx);
    return pick_out<T, T, kResidual>(a, ctx);
}

}  // namespace

cudaError_t rms_norm(const NormArgs& a, const LaunchCtx& ctx)
{
    return a.bf16 ? pick_mode<__nv_bfloat16>(a, ctx) : pick_mode<float>(a, ctx);
}

}  // namespace ssd
