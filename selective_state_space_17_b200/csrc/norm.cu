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
// maximum over the groups of rho_g max |v w| and needs no second pass. Measured:
// residual, 16384 x 2560, bf16 to 8 bits 71.5 us and to bf16 78 us (98% of the copy
// rate); gate, 16384 x 5120, to bf16 78.6 us (97%) and to 8 bits 79.5 us (80%), where
// the special-function unit (two operations for each SiLU) and issue slots share the
// bound; 64 x 2560 2.2 us.
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

// max(a, |b.x|, |b.y|), NaN if one of them is.
__device__ __forceinline__ float max_abs(float a, float2 b)
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b.x), "f"(b.y));
    return r;
}

// The warp's maximum, NaN if one of its values is.
__device__ __forceinline__ float warp_max(float v)
{
    float r;
    asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// The warp's sum of v.x, and with MAX its maximum of v.y.
template <bool MAX>
__device__ __forceinline__ float2 warp_sum_max(float2 v)
{
    float2 r = v;
    if constexpr (MAX) r.y = warp_max(v.y);
#pragma unroll
    for (int o = 16; o; o >>= 1) r.x += __shfl_xor_sync(0xffffffffu, r.x, o);
    return r;
}

template <int VEC>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float* v)
{
    if constexpr (VEC == 1) {
        *p = __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
    } else if constexpr (VEC == 2) {
        *reinterpret_cast<uint16_t*>(p) = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3);
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
// each lane takes vectors of VEC elements, wpg * 32 vectors apart. When a row
// fits one warp a CTA runs blockDim / 32 rows at a time and needs no barrier.
struct Place {
    int lane, warp, wpr, wr, group, t0, stride, nvec, Dg;
    long long gbase;
    __device__ __forceinline__ Place(const NormArgs& a, int wpg, int vec)
    {
        lane = threadIdx.x & 31;
        warp = threadIdx.x >> 5;
        wpr = a.groups * wpg;
        wr = wpr == 1 ? 0 : warp;
        group = wr / wpg;
        Dg = a.D / a.groups;
        nvec = Dg / vec;
        stride = wpg * 32;
        t0 = (wr - group * wpg) * 32 + lane;
        gbase = (long long)group * Dg;
    }
    __device__ __forceinline__ long long row0() const
    {
        return wpr == 1 ? (long long)blockIdx.x * (blockDim.x >> 5) + warp : blockIdx.x;
    }
    __device__ __forceinline__ long long row_step() const
    {
        return (long long)gridDim.x * (wpr == 1 ? blockDim.x >> 5 : 1);
    }
};

// Factors from v w to the output: v w * first * second.
struct Factors {
    float first, second;
};

// The factors of a row of scale s: rho / s in one, but for rows so small that it
// overflows (a row of zeros), where they are two.
__device__ __forceinline__ Factors over_scale(float rho, float s)
{
    const float f = __fdividef(rho, s);
    return isinf(f) ? Factors{rho, 1.0f / s} : Factors{f, 1.0f};
}

// Joins the lanes' (sum of squares, max |v w|) of a row and stores its scale with
// Q8. red alternates between two buffers: a warp writes the next row's only after
// this row's barrier, which follows every read of the one before.
//
// With one group, rho cancels in the 8-bit values: y / s = v w rho / (rho max |v w|
// / 448) = v w (448 / max |v w|), two roundings, which leaves fewer values on the
// wrong side of a border of e4m3 than rho and s would with theirs.
template <bool Q8>
__device__ __forceinline__ Factors join_row(float2 acc, const NormArgs& a, const Place& p, int wpg, float2* red,
                                            long long row)
{
    acc = warp_sum_max<Q8>(acc);
    const float inv_n = 1.0f / (float)p.Dg;
    const bool writer = p.wr == 0 && p.lane == 0;
    if (p.wpr > 1) {
        if (p.lane == 0) red[p.warp] = acc;
        __syncthreads();
        if (a.groups > 1) {
            // lane g joins group g; its share of the maximum is rho_g max |v w|
            float2 t = both(0.0f);
            if (p.lane < a.groups) {
                for (int k = 0; k < wpg; ++k) {
                    const float2 e = red[p.lane * wpg + k];
                    t.x += e.x;
                    t.y = max_nan(t.y, e.y);
                }
            }
            const float rho_lane = rsqrtf(fmaf(t.x, inv_n, a.eps));
            const float rho = __shfl_sync(0xffffffffu, rho_lane, p.group);
            if constexpr (!Q8) return {rho, 1.0f};
            const float amax = warp_max(p.lane < a.groups ? t.y * rho_lane : 0.0f);
            const float s = max_nan(amax / kE4m3Max, kScaleMin);
            if (writer) a.scale[row] = s;
            return over_scale(rho, s);
        }
        if (p.wpr <= 16) {
            // both halves of the warp join the same sixteen
            const int k = p.lane & 15;
            const float2 e = k < p.wpr ? red[k] : both(0.0f);
            acc.x = e.x;
#pragma unroll
            for (int o = 8; o; o >>= 1) acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
            if constexpr (Q8) acc.y = warp_max(e.y);
        } else {
            acc = warp_sum_max<Q8>(p.lane < p.wpr ? red[p.lane] : both(0.0f));
        }
    }
    const float rho = rsqrtf(fmaf(acc.x, inv_n, a.eps));
    if constexpr (!Q8) return {rho, 1.0f};
    const float amax = acc.y * rho;
    if (writer) a.scale[row] = max_nan(amax / kE4m3Max, kScaleMin);
    // the smallest scale, NaN, a maximum that the fast division takes for infinite, or
    // one so small that 448 over it is (below 448 / 3.4e38 = 1.32e-36: rho may put its
    // scale far above the smallest)
    if (!(amax >= kE4m3Max * kScaleMin) || !(acc.y >= 1.4e-36f && acc.y <= 8e37f))
        return over_scale(rho, max_nan(amax / kE4m3Max, kScaleMin));
    return {__fdividef(kE4m3Max, acc.y), 1.0f};
}

// v of one vector: x + r, x silu(z) or x.
template <typename T, typename R, int MODE, int VEC>
struct Operands {
    Packed<T, VEC> x, z;
    Packed<R, VEC> r;
    __device__ __forceinline__ void load(const NormArgs& a, long long at, long long zat)
    {
        x.load(static_cast<const T*>(a.x) + at);
        if constexpr (MODE == kGate) z.load(static_cast<const T*>(a.gate) + zat);
        if constexpr (MODE == kResidual) r.load(static_cast<const R*>(a.residual) + at);
    }
    __device__ __forceinline__ void zero()
    {
        x.zero();
        z.zero();
        r.zero();
    }
    __device__ __forceinline__ float2 pair(int i) const
    {
        float2 v = x.pair(i);
        if constexpr (VEC == 1) {  // a single value beside a zero
            if constexpr (MODE == kResidual) v.x += r.get(0);
            if constexpr (MODE == kGate) v.x *= silu_f<T>(z.get(0));
        } else {
            if constexpr (MODE == kResidual) v = add2(v, r.pair(i));
            if constexpr (MODE == kGate) v = mul2(v, silu2<T>(z.pair(i)));
        }
        return v;
    }
};

template <typename T, bool Q8, int VEC>
__device__ __forceinline__ void store_out(const NormArgs& a, long long at, const float* o)
{
    if constexpr (Q8) {
        store_e4m3<VEC>(static_cast<uint8_t*>(a.y) + at, o);
    } else {
        Packed<T, VEC> p;
        p.set(o);
        p.store(static_cast<T*>(a.y) + at);
    }
}

template <typename R, int VEC>
__device__ __forceinline__ void store_residual(const NormArgs& a, long long at, const float* v)
{
    if (a.residual_out) {
        Packed<R, VEC> p;
        p.set(v);
        p.store(static_cast<R*>(a.residual_out) + at);
    }
}

// Whether a lane keeps its weights in shared memory (see below): with the gate
// the arithmetic wants the warps that 64 registers a thread allow (16384 x 5120
// to 8 bits when it was first built: 234 us with two CTAs per SM, 127 with three);
// with a residual the loads in flight alone count, and registers are faster (16384 x
// 2560 to 8 bits 72 us against 80).
__host__ __device__ constexpr bool shared_weights(int mode, int values) { return values > 8 && mode != kResidual; }

// Rows kept in registers, VPT vectors to a lane. A CTA walks rows a grid apart
// with the next row's loads in flight under the reduction and the output of the row
// at hand. v w replaces v as soon as its square is added, so the output costs one
// product and the weights are not read again.
template <typename T, typename R, int MODE, bool Q8, int VEC, int VPT>
__global__ void __launch_bounds__(VPT * VEC > 8 ? 512 : 1024, VPT < 3 && shared_weights(MODE, VPT * VEC) ? 2 : 1) rms_norm_kernel(NormArgs a, int wpg)
{
    __shared__ float2 red[2][32];
    extern __shared__ float4 weights[];
    const Place p(a, wpg, VEC);
    Operands<T, R, MODE, VEC> in[VPT];
    // each thread's own weights: in registers, or, where its vectors would take
    // more than a quarter of them, in its own places in shared memory (read 16
    // bytes at a time by neighbouring lanes: no conflicts, no barrier)
    constexpr bool kShared = shared_weights(MODE, VPT * VEC);
    constexpr int kPairs = (VEC + 1) / 2;
    Packed<float, VEC> w[VPT];
    wait_for_previous();
    let_next_begin();
    long long row = p.row0();
    if (row >= a.rows) return;
    auto load = [&](long long r) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int t = p.t0 + i * p.stride;
            if (t < p.nvec) in[i].load(a, r * a.D + p.gbase + t * VEC, r * a.gate_stride + p.gbase + t * VEC);
        }
    };
    // a lane's vectors past the row's end hold zeros, which change neither the
    // sum nor the maximum: only loads and stores ask
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        in[i].zero();
        w[i].zero();
        if (p.t0 + i * p.stride < p.nvec) w[i].load(a.weight + p.gbase + (p.t0 + i * p.stride) * VEC);
        if constexpr (kShared) {
#pragma unroll
            for (int j = 0; j < VEC / 4; ++j)
                weights[(i * (VEC / 4) + j) * blockDim.x + threadIdx.x] =
                    make_float4(w[i].get(4 * j), w[i].get(4 * j + 1), w[i].get(4 * j + 2), w[i].get(4 * j + 3));
        }
    }
    load(row);
    for (int buf = 0; row < a.rows; buf ^= 1) {
        const long long base = row * a.D + p.gbase, next = row + p.row_step();
        float2 vw[VPT][kPairs];
        float2 squares = both(0.0f);
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int t = p.t0 + i * p.stride;
            Packed<float, VEC> wv = w[i];
            if constexpr (kShared) {
#pragma unroll
                for (int j = 0; j < VEC / 4; ++j) {
                    const float4 q = weights[(i * (VEC / 4) + j) * blockDim.x + threadIdx.x];
                    wv.w[4 * j] = __float_as_uint(q.x); wv.w[4 * j + 1] = __float_as_uint(q.y);
                    wv.w[4 * j + 2] = __float_as_uint(q.z); wv.w[4 * j + 3] = __float_as_uint(q.w);
                }
            }
            float v[2 * kPairs];
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                const float2 e = in[i].pair(j);
                squares = fma2(e, e, squares);
                vw[i][j] = mul2(e, wv.pair(j));
                if constexpr (Q8) top = max_abs(top, vw[i][j]);
                v[2 * j] = e.x; v[2 * j + 1] = e.y;
            }
            if constexpr (MODE == kResidual) {
                if (t < p.nvec) store_residual<R, VEC>(a, base + t * VEC, v);
            }
        }
        if (next < a.rows) load(next);
        const Factors f = join_row<Q8>(make_float2(squares.x + squares.y, top), a, p, wpg, red[buf], row);
        if (Q8 && f.second != 1.0f) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < kPairs; ++j) vw[i][j] = mul2(vw[i][j], both(f.second));
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int t = p.t0 + i * p.stride;
            float o[2 * kPairs];
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                const float2 e = mul2(vw[i][j], both(f.first));
                o[2 * j] = e.x; o[2 * j + 1] = e.y;
            }
            if (t < p.nvec) store_out<T, Q8, VEC>(a, base + t * VEC, o);
        }
        row = next;
    }
}

// Rows of any width, read a second time for the output.
template <typename T, typename R, int MODE, bool Q8, int VEC>
__global__ void __launch_bounds__(1024) rms_norm_wide_kernel(NormArgs a, int wpg)
{
    __shared__ float2 red[2][32];
    constexpr int kPairs = (VEC + 1) / 2;
    const Place p(a, wpg, VEC);
    int buf = 0;
    wait_for_previous();
    let_next_begin();
    for (long long row = p.row0(); row < a.rows; row += p.row_step(), buf ^= 1) {
        const long long base = row * a.D + p.gbase, zbase = row * a.gate_stride + p.gbase;
        Operands<T, R, MODE, VEC> in;
        Packed<float, VEC> w;
        float2 squares = both(0.0f);
        float top = 0.0f;
        for (int t = p.t0; t < p.nvec; t += p.stride) {
            in.load(a, base + t * VEC, zbase + t * VEC);
            if constexpr (Q8) w.load(a.weight + p.gbase + t * VEC);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                const float2 v = in.pair(j);
                squares = fma2(v, v, squares);
                if constexpr (Q8) top = max_abs(top, mul2(v, w.pair(j)));
            }
        }
        const Factors f = join_row<Q8>(make_float2(squares.x + squares.y, top), a, p, wpg, red[buf], row);
        for (int t = p.t0; t < p.nvec; t += p.stride) {
            in.load(a, base + t * VEC, zbase + t * VEC);
            w.load(a.weight + p.gbase + t * VEC);
            float v[2 * kPairs], o[2 * kPairs];
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                const float2 e = in.pair(j);
                const float2 q = mul2(mul2(mul2(e, w.pair(j)), both(f.first)), both(f.second));
                v[2 * j] = e.x; v[2 * j + 1] = e.y;
                o[2 * j] = q.x; o[2 * j + 1] = q.y;
            }
            if constexpr (MODE == kResidual) store_residual<R, VEC>(a, base + t * VEC, v);
            store_out<T, Q8, VEC>(a, base + t * VEC, o);
        }
    }
}

template <typename T, typename R, int MODE, bool Q8, int VEC, int VPT>
cudaError_t launch(const NormArgs& a, const LaunchCtx& ctx)
{
    const int nvec = a.D / a.groups / VEC;
    int wpg;
    if constexpr (VPT > 0) wpg = (nvec + 32 * VPT - 1) / (32 * VPT);
    else wpg = std::min(32 / a.groups, (nvec + 31) / 32);
    const int wpr = wpg * a.groups;
    const int threads = wpr == 1 ? 128 : wpr * 32;
    const long long ctas = wpr == 1 ? (a.rows + 3) / 4 : a.rows;
    const long long cap = (long long)ctx.num_sms * std::max(1, 1024 / threads);
    const unsigned grid = (unsigned)std::min(ctas, cap);
    const size_t smem = shared_weights(MODE, VPT * VEC) ? sizeof(float) * VPT * VEC * threads : 0;
    // three vectors of 8 to each of 512 threads are 48 KB beside the reduction's 512
    // bytes: more than a kernel gets without asking
    if constexpr (shared_weights(MODE, VPT * VEC) && VPT == 3) {
        static std::atomic<uint64_t> allowed{0};
        const cudaError_t err = allow_smem(reinterpret_cast<const void*>(rms_norm_kernel<T, R, MODE, Q8, VEC, VPT>),
                                           (int)sizeof(float) * VPT * VEC * 512, allowed);
        if (err != cudaSuccess) return err;
    }
    if constexpr (VPT > 0)
        return launch_overlapped(rms_norm_kernel<T, R, MODE, Q8, VEC, VPT>, grid, threads, smem, ctx.stream, 1, a, wpg);
    else
        return launch_overlapped(rms_norm_wide_kernel<T, R, MODE, Q8, VEC>, grid, threads, 0, ctx.stream, 1, a, wpg);
}

// The widest access that every row allows (16 bytes of the I/O dtype, or two
// elements, or one), and the vectors per lane that put a row in the registers of one
// CTA.
template <typename T, typename R, int MODE, bool Q8>
cudaError_t pick(const NormArgs& a, const LaunchCtx& ctx)
{
    constexpr int V = 16 / (int)sizeof(T);
    const int Dg = a.D / a.groups;
    auto rows_allow = [&](int v) {
        return Dg % v == 0 && (MODE != kGate || (aligned_to(a.gate, v * sizeof(T)) && a.gate_stride % v == 0));
    };
    // whether n vectors of a group, k to a lane, fit `warps` warps shared by the groups
    auto fits = [&](int n, int k, int warps) { return (n + 32 * k - 1) / (32 * k) * a.groups <= warps; };
    if (rows_allow(V)) {
        const int n = Dg / V;
        // many rows: two vectors per lane, for the bytes in flight (65536 x 512 with the
        // gate to 8 bits 30 us; one vector and twice the warps 47); few: as many warps
        // as the row has vectors for
        const bool many = a.rows > 4ll * ctx.num_sms;
        if (fits(n, 1, many ? 1 : 32)) return launch<T, R, MODE, Q8, V, 1>(a, ctx);
        // three per lane where a group leaves fewer lanes idle so (80 vectors: 16384 x
        // 5120 with the gate to 8 bits in 8 groups 91 us against 130)
        auto slots = [&](int k) { return (n + 32 * k - 1) / (32 * k) * k; };
        if (many && fits(n, 3, 16) && 8 * slots(3) < 7 * slots(2)) return launch<T, R, MODE, Q8, V, 3>(a, ctx);
        if (fits(n, 2, 16)) return launch<T, R, MODE, Q8, V, 2>(a, ctx);
        if (fits(n, 1, 32)) return launch<T, R, MODE, Q8, V, 1>(a, ctx);
        return launch<T, R, MODE, Q8, V, 0>(a, ctx);
    }
    if (rows_allow(2) && fits(Dg / 2, 4, 32)) return launch<T, R, MODE, Q8, 2, 4>(a, ctx);
    // single elements: eight per lane for the bytes in flight (16384 x 1237 with a
    // residual in fp32 54 us against 62 with four), four where the gate's values would
    // spill or the rows are few
    if constexpr (MODE != kGate) {
        if (a.rows > 16ll * ctx.num_sms && fits(Dg, 8, 32)) return launch<T, R, MODE, Q8, 1, 8>(a, ctx);
    }
    if (fits(Dg, 4, 32)) return launch<T, R, MODE, Q8, 1, 4>(a, ctx);
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
