// layer.cuh — arguments and launchers of the operators around the SSD core
// (norm.cu, conv.cu, linear.cu) as layer_api.cu calls them, and the device
// helpers they share.
#pragma once

#include <cuda_fp8.h>

#include <atomic>

#include "common.cuh"

namespace ssd {

// Root-mean-square norm (norm.cu). Exactly one of residual and gate may be set.
struct NormArgs {
    const void* x;          // [rows, D], I/O dtype
    const void* residual;   // [rows, D] in res_f32 ? fp32 : I/O dtype, or null
    const void* gate;       // row r at gate + r * gate_stride, I/O dtype, or null
    long long gate_stride;  // elements
    const float* weight;    // [D]
    void* y;                // [rows, D], e4m3 when scale is set, else the I/O dtype
    float* scale;           // [rows], or null
    void* residual_out;     // as residual, or null
    long long rows;
    int D, groups;
    float eps;
    bool bf16, res_f32;
};
cudaError_t rms_norm(const NormArgs& a, const LaunchCtx& ctx);

// Short causal convolution (conv.cu).
struct ConvArgs {
    const void* u;           // token t of row b at u + b * u_batch + t * u_row
    long long u_batch, u_row;
    const float* weight;     // [C, W]
    const float* bias;       // [C] or null
    const void* dt_raw;      // [.., H] beside u, or null
    long long dt_batch, dt_row;
    const float* dt_bias;    // [H] or null
    const void* init;        // [B, W-1, C] or null (zeros)
    void* x;                 // [B, L, XC]
    void* Bm;                // [B, L, GN]
    void* Cm;                // [B, L, GN]
    float* dt;               // [B, L, H]
    void* final_state;       // [B, W-1, C] or null; may be init when L == 1
    int B, L, H, XC, GN, W;
    bool silu, bf16;
    __host__ __device__ int C() const { return XC + 2 * GN; }
};
cudaError_t conv_forward(const ConvArgs& a, const LaunchCtx& ctx);

// Matrix product with its epilogue (linear.cu, linear_simt.cu).
enum class LinearType { f32, bf16, e4m3 };
struct LinearArgs {
    const void* x;         // row m at x + m * x_stride
    long long x_stride;    // elements
    const void* w;         // [N, K]
    const float* x_scale;  // [M] or null
    const float* w_scale;  // [N] or null
    const float* bias;     // [N] or null
    const void* residual;  // [M, N] in the output's dtype, or null
    void* y;               // [M, N] fp32 or bf16
    int M, N, K;
    int act;               // ssd_activation
    LinearType type;
    bool out_bf16;
};
// Bytes of workspace linear() needs for these operands (0 for most).
size_t linear_workspace_bytes(const LinearArgs& a);
cudaError_t linear(const LinearArgs& a, void* workspace, const LaunchCtx& ctx);

// Any operands; with only_if, only when that word is not zero (linear_simt.cu).
cudaError_t linear_simt(const LinearArgs& a, const unsigned int* only_if, const LaunchCtx& ctx);
// Few tokens, any operands.
cudaError_t linear_rows(const LinearArgs& a, const LaunchCtx& ctx);
// Rows of K elements copied to a pitch (elements) that TMA can address, zeros behind them.
cudaError_t pack_rows(const void* src, long long stride, int rows, int K, LinearType type, void* dst, int pitch,
                      const LaunchCtx& ctx);
// Rows of K fp32 as three sections of bf16 each; *flag = 1 if a value does not split.
cudaError_t split_rows(const float* src, long long stride, int rows, int K, void* dst, int section,
                       unsigned int* flag, const LaunchCtx& ctx);
void set_linear_variant(int variant);

// Lets a kernel take up to `bytes` of dynamic shared memory on the current
// device; `done`, one per kernel and size, holds the devices asked already.
inline cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (done.load(std::memory_order_relaxed) >> (dev & 63) & 1)) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
    return e;
}

inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// Programmatic dependent launch: a kernel launched by launch_overlapped may begin
// while the one before it on the stream ends. Every thread waits here for that
// one (all of it, and its writes) before it touches global memory.
// Such a kernel reads with plain loads: the one before may have written any operand (the
// norm the product's row scales), and a load by way of the read-only cache is for memory
// that no one writes while the kernel runs, from before this wait on.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// From here on the next kernel's CTAs may take the room this kernel leaves, once
// every CTA of this kernel has come here. Called after what a CTA takes of its SM
// for itself (tensor memory): the next kernel's CTAs hold theirs while they wait.
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename T> struct same { using type = T; };  // its argument is not deduced
template <typename T> using same_t = typename same<T>::type;

template <typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Args...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                              int cluster, const same_t<Args>&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = cluster;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// v * sigmoid(v) for an output of type O.
//
// fp32: v / (1 + e^-v), for v < 0 as v e^v / (1 + e^v), which neither overflows nor
// ends before the result leaves fp32's range; CUDA's expf, and the reciprocal of a
// value in [1, 2] off by one unit of 2^-23. Measured 7e-8 rms everywhere, and 49.8 us
// instead of 46.8 for a convolution of 4 x 2048 x 4480. (The hardware's 2^x with its
// exponent's rounding made up for, in packed instructions: 9e-8 and 56.5 us.)
//
// bf16: v / (1 + 2^(-v log2 e)) by the hardware's 2^x and 1/x, off by 2 and 1 units of
// 2^-23, and by |v| units of 2^-24 for the exponent's rounding: nothing beside bf16's.
// Below v = -87.3, where the result is under 1.1e-36 in size, the reciprocal of a
// number above 2^126 is 0, and so is the result.
template <typename O>
__device__ __forceinline__ float silu_f(float v)
{
    float p, r;
    if constexpr (sizeof(O) == 4) {
        p = expf(-fabsf(v));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + p));
        return (v < 0.0f ? v * p : v) * r;
    } else {
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(v * -1.4426950408889634f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + p));
        return v * r;
    }
}

// Two fp32 lanes in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

template <typename O>
__device__ __forceinline__ float2 silu2(float2 v)
{
    if constexpr (sizeof(O) == 4) {
        return make_float2(silu_f<O>(v.x), silu_f<O>(v.y));
    } else {
        float2 p = mul2(v, both(-1.4426950408889634f)), r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p.x) : "f"(p.x));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p.y) : "f"(p.y));
        p = add2(p, both(1.0f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(p.x));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(p.y));
        return mul2(v, r);
    }
}

// v (1 + erf(v / sqrt 2)) / 2 for an output of type O. With x = |v| / sqrt 2, q = erfc(x) / 2
// is e^(-x^2) times a function of t = 1 / (1 + 0.42 x) that stays smooth as x grows, so the
// result, v (1 - q) or for v < 0 v q, keeps its relative precision in the tail, where
// 1 + erf cancels. The function as t (c1 + c2 t + ...), the coefficients by weighted least
// squares for the smallest largest relative error over 0 <= x <= 9.5: eight of them, 1.7e-7,
// for bf16 (measured 2e-7 rms for v > -3.5, 1e-6 for v > -8; its rounding is 2e-3), ten,
// 2.3e-9, for fp32, where t takes one Newton step and the rounding of the power's exponent is
// made up for (measured 1.1e-7 rms at most over -12 to 4, 4096 x 2560 x 512 29.3 us; erfcf
// 0.7e-7 to 31e-7 and 39 us).
template <typename O>
__device__ __forceinline__ float gelu_f(float v)
{
    const float d = fmaf(fabsf(v), 0.42f * 0.70710678118654752f, 1.0f);
    constexpr float kExp = -0.5f * 1.4426950408889634f;  // -log2(e) / 2 and 9.6e-9 more
    const float h = v * v, x = h * kExp;
    float t, e, q;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(d));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
    if constexpr (sizeof(O) == 4) {
        // lost: the bits of the exponent that x has no room for. With e = 0 (v v may be
        // infinite) the result does not depend on either.
        const float lost = fmaf(h, -9.62981495e-9f, fmaf(fmaf(v, v, -h), kExp, fmaf(h, kExp, -x)));
        if (e > 0.0f) {
            t = fmaf(t, fmaf(-d, t, 1.0f), t);
            e = fmaf(e, lost * 0.69314718f, e);
        }
        q = fmaf(t, 0.5f * -0.0411372973f, 0.5f * 0.2307045f);
        q = fmaf(q, t, 0.5f * -0.486641164f);
        q = fmaf(q, t, 0.5f * 0.437147986f);
        q = fmaf(q, t, 0.5f * -0.197327718f);
        q = fmaf(q, t, 0.5f * 0.213732748f);
        q = fmaf(q, t, 0.5f * 0.150040975f);
        q = fmaf(q, t, 0.5f * 0.21989442f);
        q = fmaf(q, t, 0.5f * 0.236612227f);
        q = fmaf(q, t, 0.5f * 0.236973321f);
    } else {
        q = fmaf(t, 0.5f * 0.0702151842f, 0.5f * -0.320189623f);
        q = fmaf(q, t, 0.5f * 0.440556504f);
        q = fmaf(q, t, 0.5f * -0.130418142f);
        q = fmaf(q, t, 0.5f * 0.268684546f);
        q = fmaf(q, t, 0.5f * 0.194744036f);
        q = fmaf(q, t, 0.5f * 0.239582894f);
        q = fmaf(q, t, 0.5f * 0.236824431f);
    }
    q = q * t * e;
    return v * (v >= 0.0f ? 1.0f - q : q);
}

template <typename O>
__device__ __forceinline__ float activate(float v, int act)
{
    if (act == SSD_ACT_SILU) return silu_f<O>(v);
    if (act == SSD_ACT_GELU) return gelu_f<O>(v);
    return v;
}

// VEC consecutive elements of type T as they lie in memory (one access of up
// to 16 bytes each, two for 32 bytes), and as fp32 values.
template <typename T, int VEC>
struct Packed {
    static constexpr int kBytes = VEC * (int)sizeof(T);
    static constexpr int kWords = kBytes >= 4 ? kBytes / 4 : 1;
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const T* p)
    {
        if constexpr (kBytes >= 16) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i) {
                const uint4 v = *(reinterpret_cast<const uint4*>(p) + i);
                w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
            }
        } else if constexpr (kBytes == 8) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            w[0] = v.x; w[1] = v.y;
        } else if constexpr (kBytes == 4) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
            w[0] = *reinterpret_cast<const uint16_t*>(p);
        }
    }
    __device__ __forceinline__ void store(T* p) const
    {
        if constexpr (kBytes >= 16) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i)
                *(reinterpret_cast<uint4*>(p) + i) =
                    make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else if constexpr (kBytes == 8) {
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        } else if constexpr (kBytes == 4) {
            *reinterpret_cast<uint32_t*>(p) = w[0];
        } else {
            *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
        }
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float((i & 1) ? (w[i / 2] & 0xFFFF0000u) : (w[i / 2] << 16));
    }
    // elements 2i and 2i + 1 (0 beside a single one)
    __device__ __forceinline__ float2 pair(int i) const
    {
        if constexpr (VEC == 1) return make_float2(get(0), 0.0f);
        else return make_float2(get(2 * i), get(2 * i + 1));
    }
    __device__ __forceinline__ void set(const float* v)
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) w[i] = __float_as_uint(v[i]);
        } else if constexpr (VEC == 1) {
            w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
        } else {
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
        }
    }
};

}  // namespace ssd
