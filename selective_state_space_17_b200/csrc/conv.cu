// conv.cu — short causal convolution over each channel, with SiLU, that cuts
// the in-projection's rows into the SSD core's operands:
//
//     v[t, c] = bias[c] + sum_k weight[c, k] u[t - W + 1 + k, c]
//     (x | B | C)[t] = silu(v[t]),   dt[t, h] = softplus(raw[t, h] + dt_bias[h])
//
// with the W - 1 tokens before token 0 taken from a state (zeros without one).
// Bound by HBM: each input element is read once and each output written once.
// A thread walks a strip of tokens of VEC neighbouring channels (one 16-byte
// access per token) with the window's W - 1 older inputs and the channels'
// W weights in registers, so a strip reads its tokens and W - 1 more; strips of
// one channel lie in one CTA column and their overlap hits L2. The single-token
// form is the same kernel with one token per strip; it loads its whole window
// at once and may write the state in place.
#include <algorithm>

#include "layer.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 4;  // tokens loaded before the first of them is used

__device__ __forceinline__ float softplus_f(float v)
{
    // log(1 + e^v) = max(v, 0) + log(1 + e^-|v|): no overflow at either end
    return fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v)));
}

template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kThreads) conv_kernel(ConvArgs a, int strip, int channel_ctas)
{
    const int b = blockIdx.z;
    const int t0 = blockIdx.y * strip, t1 = min(t0 + strip, a.L);
    if ((int)blockIdx.x >= channel_ctas) {
        // step sizes of this strip's tokens
        const T* raw = static_cast<const T*>(a.dt_raw) + b * a.dt_batch;
        const long long n = (long long)(t1 - t0) * a.H;
        const int step = ((int)gridDim.x - channel_ctas) * kThreads;
        for (long long i = ((int)blockIdx.x - channel_ctas) * kThreads + threadIdx.x; i < n; i += step) {
            const int t = t0 + (int)(i / a.H), h = (int)(i % a.H);
            float v = io<T>::load(raw + t * a.dt_row + h);
            if (a.dt_bias) v += __ldg(a.dt_bias + h);
            a.dt[((long long)b * a.L + t) * a.H + h] = softplus_f(v);
        }
        return;
    }
    const int C = a.C();
    const int c = ((int)blockIdx.x * kThreads + threadIdx.x) * VEC;
    if (c >= C) return;
    const T* u = static_cast<const T*>(a.u) + b * a.u_batch + c;
    const T* init = static_cast<const T*>(a.init) + (long long)b * (W - 1) * C + c;
    // the output section of these channels (sections are multiples of VEC)
    T* out;
    int width;
    if (c < a.XC) {
        out = static_cast<T*>(a.x) + c;
        width = a.XC;
    } else if (c < a.XC + a.GN) {
        out = static_cast<T*>(a.Bm) + (c - a.XC);
        width = a.GN;
    } else {
        out = static_cast<T*>(a.Cm) + (c - a.XC - a.GN);
        width = a.GN;
    }
    out += ((long long)b * a.L + t0) * width;

    // the window: win[k] is input t - (W - 1) + k of the token t at hand
    Packed<T, VEC> win[W - 1 + kAhead];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const int t = t0 - (W - 1) + k;
        win[k].zero();
        if (t >= 0) win[k].load(u + t * a.u_row);
        else if (a.init) win[k].load(init + (long long)(t + W - 1) * C);
    }
    Packed<float, VEC * W> wt;  // weight of channel j, tap k: element j W + k
    Packed<float, VEC> bias;
    if constexpr (VEC > 1) {
        wt.load(a.weight + (long long)c * W);
    } else {
#pragma unroll
        for (int k = 0; k < W; ++k) wt.w[k] = __float_as_uint(a.weight[(long long)c * W + k]);
    }
    bias.zero();
    if (a.bias) bias.load(a.bias + c);
    for (int t = t0; t < t1; t += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            win[W - 1 + i].zero();
            if (t + i < t1) win[W - 1 + i].load(u + (long long)(t + i) * a.u_row);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (t + i >= t1) break;
            float v[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                v[j] = bias.get(j);
#pragma unroll
                for (int k = 0; k < W; ++k) v[j] = fmaf(wt.get(j * W + k), win[i + k].get(j), v[j]);
                if (a.silu) v[j] = silu_f(v[j]);
            }
            Packed<T, VEC> o;
            o.set(v);
            o.store(out);
            out += width;
        }
        // keep the last W - 1 inputs; after the last group, those of token t1 - 1
        const int n = min(kAhead, t1 - t);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            Packed<T, VEC> keep = win[k];
#pragma unroll
            for (int i = 1; i <= kAhead; ++i)
                if (n == i) keep = win[k + i];
            win[k] = keep;
        }
    }
    if (a.final_state && t1 == a.L) {
        T* fs = static_cast<T*>(a.final_state) + (long long)b * (W - 1) * C + c;
#pragma unroll
        for (int k = 0; k < W - 1; ++k) win[k].store(fs + (long long)k * C);
    }
}

template <typename T, int VEC, int W>
cudaError_t launch(const ConvArgs& a, const LaunchCtx& ctx)
{
    const int cx = (a.C() / VEC + kThreads - 1) / kThreads;
    // strips as long as leave about eight CTAs per SM, and 64 tokens at most
    const long long want = (8ll * ctx.num_sms + (long long)cx * a.B - 1) / ((long long)cx * a.B);
    int strip = (int)std::max(1ll, std::min<long long>(64, a.L / want));
    strip = std::max(strip, (a.L + 65534) / 65535);  // the grid's y extent
    strip = (strip + kAhead - 1) / kAhead * kAhead;
    const int strips = (a.L + strip - 1) / strip;
    const long long steps = (long long)a.H * std::min(strip, a.L);  // step sizes of a strip
    const int dx = a.dt_raw ? (int)std::max(1ll, std::min(steps / (4 * kThreads), 8ll)) : 0;
    conv_kernel<T, VEC, W><<<dim3(cx + dx, (unsigned)strips, a.B), kThreads, 0, ctx.stream>>>(a, strip, cx);
    return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t pick_width(const ConvArgs& a, const LaunchCtx& ctx)
{
    if (a.W == 2) return launch<T, VEC, 2>(a, ctx);
    if (a.W == 3) return launch<T, VEC, 3>(a, ctx);
    return launch<T, VEC, 4>(a, ctx);
}

template <typename T>
cudaError_t pick(const ConvArgs& a, const LaunchCtx& ctx)
{
    constexpr int V = 16 / (int)sizeof(T);
    const bool vec = a.XC % V == 0 && a.GN % V == 0 && aligned_to(a.u, 16) && a.u_row % V == 0 &&
                     a.u_batch % V == 0;
    return vec ? pick_width<T, V>(a, ctx) : pick_width<T, 1>(a, ctx);
}

}  // namespace

cudaError_t conv_forward(const ConvArgs& a, const LaunchCtx& ctx)
{
    return a.bf16 ? pick<__nv_bfloat16>(a, ctx) : pick<float>(a, ctx);
}

}  // namespace ssd
