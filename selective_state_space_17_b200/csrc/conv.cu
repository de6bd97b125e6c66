// conv.cu — short causal convolution over each channel, with SiLU, that cuts
// the in-projection's rows into the SSD core's operands:
//
//     v[t, c] = bias[c] + sum_k weight[c, k] u[t - W + 1 + k, c]
//     (x | B | C)[t] = silu(v[t]),   dt[t, h] = softplus(raw[t, h] + dt_bias[h])
//
// with the W - 1 tokens before token 0 taken from a state (zeros without one).
// Bound by HBM: each input element is read once and each output written once.
// A thread walks a strip of tokens of VEC neighbouring channels with the
// window's inputs and the channels' W weights in registers and the next tokens'
// loads in flight, so a strip reads its tokens and W - 1 more; neighbouring
// strips run at about the same time, and their overlap hits L2. What counts is the
// bytes in flight: four channels to a thread (8 bytes of bf16) and each token's
// load eight tokens before its use measured 70 us at 4 x 4096 x 5376 in bf16,
// 5.1 TB/s, four tokens ahead 82 us, and eight channels with four tokens loaded
// before each four 118 us at 127 registers a thread. The exponentials and
// reciprocals of SiLU take 40 us of the special-function unit meanwhile. The
// single-token form is the same kernel with one token per strip; it may shift the
// state in place.
#include <algorithm>

#include "layer.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float softplus_f(float v)
{
    // log(1 + e^v) = max(v, 0) + log(1 + e^-|v|): no overflow at either end
    return fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v)));
}

// kAhead: tokens whose loads are in flight. The launch bound holds bf16 at 72
// registers a thread, seven CTAs per SM (71.5 us against 73.6 at 80 registers).
template <typename T, int VEC, int W, int kAhead>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && VEC > 1 && kAhead > 1 ? 7 : 1) conv_kernel(ConvArgs a, int strip, int channel_ctas)
{
    wait_for_previous();
    let_next_begin();
    const int b = blockIdx.z;
    const int t0 = blockIdx.y * strip, t1 = min(t0 + strip, a.L);
    if ((int)blockIdx.x >= channel_ctas) {
        // step sizes of this strip's tokens
        const T* raw = static_cast<const T*>(a.dt_raw) + b * a.dt_batch;
        // (t, h) steps by the CTAs' threads: q tokens and r heads; kBatch loads are
        // under way before the first is used
        constexpr int kBatch = 4;
        const int threads = ((int)gridDim.x - channel_ctas) * kThreads;
        const int first = ((int)blockIdx.x - channel_ctas) * kThreads + threadIdx.x;
        const int q = threads / a.H, r = threads - q * a.H;
        int t = t0 + first / a.H, h = first % a.H;
        while (t < t1) {
            T in[kBatch];
            int ts[kBatch], hs[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                ts[i] = t;
                hs[i] = h;
                if (t < t1) in[i] = raw[t * a.dt_row + h];
                t += q;
                h += r;
                if (h >= a.H) {
                    h -= a.H;
                    ++t;
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (ts[i] >= t1) break;
                float v = static_cast<float>(in[i]);
                if (a.dt_bias) v += a.dt_bias[hs[i]];
                a.dt[((long long)b * a.L + ts[i]) * a.H + hs[i]] = softplus_f(v);
            }
        }
        return;
    }
    const int C = a.C();
    const int c = ((int)blockIdx.x * kThreads + threadIdx.x) * VEC;
    if (c >= C) return;
    const T* u = static_cast<const T*>(a.u) + b * a.u_batch + c;
    const T* init = static_cast<const T*>(a.init) + (long long)b * (W - 1) * C + c;
    // the output section of these channels (a section is a multiple of VEC)
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

    constexpr int kPairs = (VEC + 1) / 2;
    // input t of these channels, or of the state before token 0
    auto input = [&](int t, Packed<T, VEC>& p) {
        p.zero();
        if (t >= 0) p.load(u + t * a.u_row);
        else if (a.init) p.load(init + (long long)(t + W - 1) * C);
    };
    // the window: win[k] is input t - (W - 1) + k of the token t at hand, in
    // fp32; next holds that token and those after it as they were read
    float2 win[W][kPairs];
    Packed<T, VEC> next[kAhead], before[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) input(t0 - (W - 1) + k, before[k]);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        next[i].zero();
        if (t0 + i < t1) input(t0 + i, next[i]);
    }
    Packed<float, VEC * W> weights;  // channel j, tap k at j W + k
    Packed<float, VEC> bias;
    if constexpr (VEC > 1) {
        weights.load(a.weight + (long long)c * W);
    } else {
#pragma unroll
        for (int k = 0; k < W; ++k) weights.w[k] = __float_as_uint(a.weight[(long long)c * W + k]);
    }
    bias.zero();
    if (a.bias) bias.load(a.bias + c);
    float2 wt[W][kPairs];
#pragma unroll
    for (int k = 0; k < W; ++k)
#pragma unroll
        for (int j = 0; j < kPairs; ++j)
            wt[k][j] = make_float2(weights.get(2 * j * W + k), VEC > 1 ? weights.get((2 * j + 1) * W + k) : 0.0f);
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
#pragma unroll
        for (int j = 0; j < kPairs; ++j) win[k][j] = before[k].pair(j);

    const T* src = u + (long long)(t0 + kAhead) * a.u_row;
    for (int left = t1 - t0; left > 0; left -= kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
#pragma unroll
            for (int j = 0; j < kPairs; ++j) win[W - 1][j] = next[i].pair(j);
            if (kAhead + i < left) next[i].load(src);
            src += a.u_row;
            float v[2 * kPairs];
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                float2 s = bias.pair(j);
#pragma unroll
                for (int k = 0; k < W; ++k) s = fma2(wt[k][j], win[k][j], s);
                if (a.silu) s = silu2<T>(s);
                v[2 * j] = s.x; v[2 * j + 1] = s.y;
#pragma unroll
                for (int k = 0; k < W - 1; ++k) win[k][j] = win[k + 1][j];
            }
            Packed<T, VEC> o;
            o.set(v);
            if (i < left) o.store(out);
            out += width;
        }
    }
    if (a.final_state && t1 == a.L) {
        // read before the first is written: the single-token form shifts the state in place
        T* fs = static_cast<T*>(a.final_state) + (long long)b * (W - 1) * C + c;
        if (a.L > 1) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k) input(a.L - (W - 1) + k, before[k]);
        } else {
#pragma unroll
            for (int k = 0; k < W - 2; ++k) before[k] = before[k + 1];
            input(0, before[W - 2]);
        }
#pragma unroll
        for (int k = 0; k < W - 1; ++k) before[k].store(fs + (long long)k * C);
    }
}

template <typename T, int VEC, int W, int kAhead>
cudaError_t launch(const ConvArgs& a, const LaunchCtx& ctx)
{
    const int cx = (a.C() / VEC + kThreads - 1) / kThreads;
    // strips as long as leave about 32 CTAs per SM, and 32 tokens at most
    const long long want = (32ll * ctx.num_sms + (long long)cx * a.B - 1) / ((long long)cx * a.B);
    int strip = (int)std::max(1ll, std::min<long long>(32, a.L / want));
    strip = std::max(strip, a.L / 65535 + 1);  // the grid's y extent
    strip = (strip + kAhead - 1) / kAhead * kAhead;
    const int strips = (a.L + strip - 1) / strip;
    const int dx = a.dt_raw ? std::max(1, std::min(a.H / 256, 8)) : 0;  // CTAs of a strip's step sizes
    return launch_overlapped(conv_kernel<T, VEC, W, kAhead>, dim3(cx + dx, strips, a.B), kThreads, 0, ctx.stream, 1, a,
                             strip, cx);
}

template <typename T, int VEC, int kAhead>
cudaError_t pick_width(const ConvArgs& a, const LaunchCtx& ctx)
{
    if (a.W == 2) return launch<T, VEC, 2, kAhead>(a, ctx);
    if (a.W == 3) return launch<T, VEC, 3, kAhead>(a, ctx);
    return launch<T, VEC, 4, kAhead>(a, ctx);
}

// One token has nothing to load ahead (64 x 5376: 4.0 us against 4.9).
template <typename T, int VEC>
cudaError_t pick_ahead(const ConvArgs& a, const LaunchCtx& ctx)
{
    return a.L == 1 ? pick_width<T, VEC, 1>(a, ctx) : pick_width<T, VEC, 8>(a, ctx);
}

template <typename T>
cudaError_t pick(const ConvArgs& a, const LaunchCtx& ctx)
{
    constexpr int V = 4;
    const bool vec = a.XC % V == 0 && a.GN % V == 0 && aligned_to(a.u, V * sizeof(T)) && a.u_row % V == 0 &&
                     a.u_batch % V == 0;
    return vec ? pick_ahead<T, V>(a, ctx) : pick_ahead<T, 1>(a, ctx);
}

}  // namespace

cudaError_t conv_forward(const ConvArgs& a, const LaunchCtx& ctx)
{
    return a.bf16 ? pick<__nv_bfloat16>(a, ctx) : pick<float>(a, ctx);
}

}  // namespace ssd
