// layer_api.cu — the C ABI of the operators around the SSD core: argument
// checks and dispatch. Declarations and contracts are in include/ssd.h.
#include <math.h>

#include "layer.cuh"

namespace ssd {
namespace {

bool io_dtype(ssd_dtype d) { return d == SSD_F32 || d == SSD_BF16; }
size_t io_size(ssd_dtype d) { return d == SSD_F32 ? 4 : 2; }

// Bytes of n rows of `width` elements, `stride` elements apart.
size_t extent(long long n, long long stride, long long width, size_t size)
{
    return n > 0 ? static_cast<size_t>((n - 1) * stride + width) * size : 0;
}

struct Span {
    const void* p;
    size_t bytes;
};
bool overlap(Span a, Span b)
{
    const char* p = static_cast<const char*>(a.p);
    const char* q = static_cast<const char*>(b.p);
    return p && q && a.bytes && b.bytes && p < q + b.bytes && q < p + a.bytes;
}
// Whether one of the outputs lies over an input or another output.
template <int NO, int NI>
bool any_overlap(const Span (&out)[NO], const Span (&in)[NI])
{
    for (int i = 0; i < NO; ++i) {
        for (const Span& s : in)
            if (overlap(out[i], s)) return true;
        for (int j = i + 1; j < NO; ++j)
            if (overlap(out[i], out[j])) return true;
    }
    return false;
}

ssd_status launched(cudaError_t e) { return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA; }

ssd_status conv_call(const void* u, long long u_batch, long long u_row, const float* weight,
                     const float* bias, const void* dt_raw, long long dt_batch, long long dt_row,
                     const float* dt_bias, const void* init, void* x, void* Bm, void* Cm, float* dt,
                     void* final_state, int B, int L, int H, int P, int G, int N, int width,
                     ssd_activation act, ssd_dtype dtype, bool step, ssd_stream_t stream)
{
    ssd_status st = check_dims(B, L, H, P, G, N, 1, dtype);
    if (st != SSD_OK) return st;
    if (width < 1 || u_batch < 0 || u_row < 0 || dt_batch < 0 || dt_row < 0) return SSD_ERR_INVALID_ARG;
    if (act != SSD_ACT_NONE && act != SSD_ACT_SILU) return SSD_ERR_INVALID_ARG;
    if (width < 2 || width > 4 || B > 65535 || L > (1 << 30)) return SSD_ERR_UNSUPPORTED;
    const bool empty = (long long)B * L == 0;
    if (!empty && (!u || !weight || !x || !Bm || !Cm)) return SSD_ERR_INVALID_ARG;
    if (!empty && ((dt_raw != nullptr) != (dt != nullptr) || (dt_bias && !dt_raw))) return SSD_ERR_INVALID_ARG;
    if (step && !empty && !init) return SSD_ERR_INVALID_ARG;
    const void* ptrs[] = {weight, bias, dt_bias, init, x, Bm, Cm, dt, final_state};
    for (const void* p : ptrs)
        if (!aligned_to(p, 16)) return SSD_ERR_MISALIGNED;
    if (!aligned_to(u, io_size(dtype)) || !aligned_to(dt_raw, io_size(dtype))) return SSD_ERR_MISALIGNED;
    ConvArgs a;
    a.u = u; a.u_batch = u_batch; a.u_row = u_row; a.weight = weight; a.bias = bias;
    a.dt_raw = dt_raw; a.dt_batch = dt_batch; a.dt_row = dt_row; a.dt_bias = dt_bias;
    a.init = init; a.x = x; a.Bm = Bm; a.Cm = Cm; a.dt = dt; a.final_state = final_state;
    a.B = B; a.L = L; a.H = H; a.XC = H * P; a.GN = G * N; a.W = width;
    a.silu = act == SSD_ACT_SILU; a.bf16 = dtype == SSD_BF16;
    // A strip of tokens may write the final state while another reads the
    // initial one: they share a buffer only in the single-token form, whose
    // threads each shift their own channels.
    const size_t es = io_size(dtype), bytes = (size_t)B * (width - 1) * a.C() * es;
    const size_t tokens = (size_t)B * L;
    if (!empty || final_state) {
        const Span out[] = {{x, tokens * a.XC * es}, {Bm, tokens * a.GN * es}, {Cm, tokens * a.GN * es},
                            {dt, tokens * H * 4}, {final_state, bytes}};
        const Span in[] = {{u, B && L ? ((B - 1) * u_batch + (L - 1) * u_row + a.C()) * es : 0},
                           {dt_raw, B && L ? ((B - 1) * dt_batch + (L - 1) * dt_row + H) * es : 0},
                           {weight, (size_t)a.C() * width * 4}, {bias, (size_t)a.C() * 4},
                           {dt_bias, (size_t)H * 4}, {step ? nullptr : init, bytes}};
        if (any_overlap(out, in)) return SSD_ERR_INVALID_ARG;
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (empty) {
        if (!final_state || bytes == 0 || step) return SSD_OK;
        return launched(init ? cudaMemcpyAsync(final_state, init, bytes, cudaMemcpyDeviceToDevice, s)
                             : cudaMemsetAsync(final_state, 0, bytes, s));
    }
    LaunchCtx ctx;
    st = acquire_launch_ctx(s, &ctx);
    if (st != SSD_OK) return st;
    return launched(conv_forward(a, ctx));
}

// The checks of a product's sizes, and what decides its path.
ssd_status linear_args(const void* x, int64_t x_stride, int M, int N, int K, ssd_dtype dtype, LinearArgs* a)
{
    if (M < 0 || N < 0 || K < 1) return SSD_ERR_INVALID_ARG;
    if (dtype != SSD_E4M3 && !io_dtype(dtype)) return SSD_ERR_INVALID_ARG;
    if (M > (1 << 30) || N > (1 << 20) || K > (1 << 20)) return SSD_ERR_UNSUPPORTED;
    a->x = x;
    a->x_stride = M > 1 ? x_stride : K;  // one row is as good as contiguous
    a->M = M;
    a->N = N;
    a->K = K;
    a->type = dtype == SSD_F32 ? LinearType::f32 : dtype == SSD_BF16 ? LinearType::bf16 : LinearType::e4m3;
    return SSD_OK;
}

}  // namespace

}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status ssd_rms_norm(const void* x, const void* residual, const void* gate, int64_t gate_stride,
                        const float* weight, void* y, float* scale, void* residual_out,
                        int64_t rows, int D, int groups, float eps, ssd_dtype dtype,
                        ssd_dtype residual_dtype, ssd_dtype y_dtype, ssd_stream_t stream)
{
    if (rows < 0 || D < 1 || groups < 1 || D % groups != 0) return SSD_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || isinf(eps)) return SSD_ERR_INVALID_ARG;
    if (!io_dtype(dtype) || (y_dtype != dtype && y_dtype != SSD_E4M3)) return SSD_ERR_INVALID_ARG;
    if (residual && residual_dtype != dtype && residual_dtype != SSD_F32) return SSD_ERR_INVALID_ARG;
    if (groups > 32 || D > (1 << 20) || rows > (1ll << 31) - 1) return SSD_ERR_UNSUPPORTED;
    if ((residual && gate) || (residual_out && !residual)) return SSD_ERR_INVALID_ARG;
    if (rows == 0) return SSD_OK;
    if (!x || !weight || !y || (y_dtype == SSD_E4M3) != (scale != nullptr)) return SSD_ERR_INVALID_ARG;
    if (gate && rows > 1 && gate_stride < D) return SSD_ERR_INVALID_ARG;
    const void* ptrs[] = {x, residual, weight, y, scale, residual_out};
    for (const void* p : ptrs)
        if (!aligned_to(p, 16)) return SSD_ERR_MISALIGNED;
    if (!aligned_to(gate, io_size(dtype))) return SSD_ERR_MISALIGNED;
    const size_t es = io_size(dtype), rs = io_size(residual_dtype), n = (size_t)rows * D;
    const bool in_place = y == x && y_dtype == dtype, same_res = residual_out == residual;
    const Span out[] = {{y, n * (y_dtype == SSD_E4M3 ? 1 : es)}, {scale, (size_t)rows * 4},
                        {residual_out, n * rs}};
    const Span in[] = {{in_place ? nullptr : x, n * es}, {same_res ? nullptr : residual, n * rs},
                       {gate, extent(rows, gate_stride, D, es)}, {weight, (size_t)D * 4}};
    if (any_overlap(out, in)) return SSD_ERR_INVALID_ARG;
    LaunchCtx ctx;
    const ssd_status st = acquire_launch_ctx(reinterpret_cast<cudaStream_t>(stream), &ctx);
    if (st != SSD_OK) return st;
    NormArgs a;
    a.x = x; a.residual = residual; a.gate = gate; a.gate_stride = gate_stride; a.weight = weight;
    a.y = y; a.scale = scale; a.residual_out = residual_out; a.rows = rows; a.D = D;
    a.groups = groups; a.eps = eps; a.bf16 = dtype == SSD_BF16; a.res_f32 = residual_dtype == SSD_F32;
    return launched(rms_norm(a, ctx));
}

size_t ssd_linear_workspace_size(const void* x, int64_t x_stride, int M, int N, int K, ssd_dtype dtype)
{
    LinearArgs a = {};
    if (M < 1 || N < 1 || linear_args(x, x_stride, M, N, K, dtype, &a) != SSD_OK) return 0;
    return linear_workspace_bytes(a);
}

ssd_status ssd_linear(const void* x, int64_t x_stride, const void* w, const float* x_scale,
                      const float* w_scale, const float* bias, const void* residual, void* y, int M,
                      int N, int K, ssd_activation act, ssd_dtype dtype, ssd_dtype y_dtype,
                      void* workspace, size_t workspace_bytes, ssd_stream_t stream)
{
    LinearArgs a = {};
    ssd_status st = linear_args(x, x_stride, M, N, K, dtype, &a);
    if (st != SSD_OK) return st;
    if (!io_dtype(y_dtype)) return SSD_ERR_INVALID_ARG;
    if (act != SSD_ACT_NONE && act != SSD_ACT_SILU && act != SSD_ACT_GELU) return SSD_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return SSD_OK;
    if (!x || !w || !y) return SSD_ERR_INVALID_ARG;
    if ((dtype == SSD_E4M3) != (x_scale != nullptr) || (dtype == SSD_E4M3) != (w_scale != nullptr))
        return SSD_ERR_INVALID_ARG;
    if (M > 1 && x_stride < K) return SSD_ERR_INVALID_ARG;
    const void* ptrs[] = {w, x_scale, w_scale, bias, residual, y, workspace};
    for (const void* p : ptrs)
        if (!aligned_to(p, 16)) return SSD_ERR_MISALIGNED;
    const size_t es = dtype == SSD_E4M3 ? 1 : io_size(dtype), ys = (size_t)M * N * io_size(y_dtype);
    if (!aligned_to(x, es)) return SSD_ERR_MISALIGNED;
    const size_t need = linear_workspace_bytes(a);
    if (need > 0 && (!workspace || workspace_bytes < need)) return SSD_ERR_WORKSPACE;
    const Span out[] = {{y, ys}, {need ? workspace : nullptr, need}};
    const Span in[] = {{x, extent(M, x_stride, K, es)}, {w, (size_t)N * K * es}, {x_scale, (size_t)M * 4},
                       {w_scale, (size_t)N * 4}, {bias, (size_t)N * 4},
                       {residual == y ? nullptr : residual, ys}};
    if (any_overlap(out, in)) return SSD_ERR_INVALID_ARG;
    LaunchCtx ctx;
    st = acquire_launch_ctx(reinterpret_cast<cudaStream_t>(stream), &ctx);
    if (st != SSD_OK) return st;
    a.w = w; a.x_scale = x_scale; a.w_scale = w_scale; a.bias = bias; a.residual = residual; a.y = y;
    a.act = act;
    a.out_bf16 = y_dtype == SSD_BF16;
    return launched(linear(a, workspace, ctx));
}

void ssd_set_linear_variant(int variant) { set_linear_variant(variant); }

ssd_status ssd_conv(const void* u, int64_t u_batch_stride, int64_t u_row_stride, const float* weight,
                    const float* bias, const void* dt_raw, int64_t dt_batch_stride,
                    int64_t dt_row_stride, const float* dt_bias, const void* initial_state, void* x,
                    void* Bm, void* Cm, float* dt, void* final_state, int B, int L, int H, int P,
                    int G, int N, int width, ssd_activation act, ssd_dtype dtype,
                    ssd_stream_t stream)
{
    return conv_call(u, u_batch_stride, u_row_stride, weight, bias, dt_raw, dt_batch_stride,
                     dt_row_stride, dt_bias, initial_state, x, Bm, Cm, dt, final_state, B, L, H, P, G,
                     N, width, act, dtype, false, stream);
}

ssd_status ssd_conv_step(const void* u, int64_t u_stride, const float* weight, const float* bias,
                         const void* dt_raw, int64_t dt_stride, const float* dt_bias, void* state,
                         void* x, void* Bm, void* Cm, float* dt, int B, int H, int P, int G, int N,
                         int width, ssd_activation act, ssd_dtype dtype, ssd_stream_t stream)
{
    return conv_call(u, u_stride, 0, weight, bias, dt_raw, dt_stride, 0, dt_bias, state, x, Bm, Cm, dt,
                     state, B, 1, H, P, G, N, width, act, dtype, true, stream);
}

}  // extern "C"
