// linear.cu — matrix product with its epilogue on the tensor cores (tcgen05),
// bf16 or e4m3 operands:
//
//     y[m, n] = act(xs[m] ws[n] sum_k x[m, k] w[n, k] + bias[n]) + residual[m, n]
//
// Two kernels. Few tokens (linear_few_kernel): the weights' bytes bound the
// call, so w takes the 128 lanes of the accumulator, the tokens its columns,
// and the K axis is cut over a cluster of CTAs that join their parts through
// distributed shared memory. Many tokens (linear_many_kernel): the tensor cores
// bound the call; persistent CTA pairs on 256-row tiles.
//
// Both stage operand rows of 128 bytes (64 bf16 or 128 e4m3 values) by TMA with
// the 128-byte swizzle; one tcgen05.mma takes 32 bytes of each row, whatever
// the type, so the two types share all but the instruction.
//
// Measured (channels x K): 64 tokens, 10576 x 2560, bf16 14.5 us (55 MB of weights:
// 3.8 TB/s), e4m3 10 us; one token, 1024 x 2048, 4.2 us; 16384 tokens, 10576 x 2560,
// in bursts bf16 600 us (1480 TFLOP/s) and e4m3 336 us (2640), in a long loop under
// the power cap 686 and 376 us; 2560 x 5120 with an fp32 residual 361 us (1190).
#include <algorithm>
#include <atomic>

#include "layer.cuh"
#include "sm100_mma.cuh"

namespace ssd {
namespace {

using namespace sm100;

std::atomic<int> g_variant{0};  // test hook: 0 automatic, 1 SIMT, 2 few tokens, 3 many tokens

constexpr int kRowBytes = 128;  // bytes of an operand row in one stage

// The K axis as the kernels walk it, in blocks of one stage: `sections` runs of
// `per` blocks; section i reads x from column x_section(i) * cols on, w likewise.
// One section for operands as they are; six for fp32 operands held as three bf16
// sections each (see linear_split).
struct Axis {
    int per, sections, cols;
    uint32_t x_sections, w_sections;  // two bits for each section
    __host__ __device__ int blocks() const { return per * sections; }
    __device__ __forceinline__ int x_col(int section) const { return (x_sections >> (2 * section) & 3) * cols; }
    __device__ __forceinline__ int w_col(int section) const { return (w_sections >> (2 * section) & 3) * cols; }
};

// Operands that TMA can address: columns and pitch in elements.
struct Operands {
    const void* x;
    const void* w;
    long long x_cols, x_pitch, w_cols, w_pitch;
    Axis axis;
    const unsigned int* skip;  // with it, nothing is computed when the word is not zero
};

struct Epilogue {
    const float* x_scale;
    const float* w_scale;
    const float* bias;
    const void* residual;
    void* y;
    int M, N, act;
};

// ------------------------------------------------------------- few tokens

// The tensor cores truncate each addition to an accumulator, a bias that grows with
// the additions in a row: after 5120 bf16 products -4.8e-6 of the result of normal
// operands and -1.8e-5 of positive ones, after 1024 -0.9e-6 and -1.7e-6. fp32 outputs
// of bf16 operands are therefore summed in segments of kSegBlocks blocks of K (768
// products), joined in registers with rounded additions: -0.6e-6 and -1.3e-6 at any K.
// A bf16 output's own rounding hides the bias, and products of e4m3 values, with
// eight significant bits at most, lose next to nothing (1e-8 at K = 5120).
constexpr int kSegBlocks = 12;

// One CTA: 128 channels x BN tokens over its part of K; eight warps that read the
// accumulators (two, in turn, when there are several segments), one that loads and
// one that issues the products. The parts of a cluster meet in shared memory: every
// CTA writes its fp32 tile there, and CTA r adds up the tokens r, r + S, ... in the
// order of the ranks, so the sum does not depend on who is first.
constexpr int kFewWarps = 8, kFewThreads = 32 * (kFewWarps + 2), kMostSplits = 8, kPrefetch = 6;

template <int V>
struct Int {
    static constexpr int value = V;
};

// DEEP: one CTA per SM with all of its shared memory, for calls of no more CTAs
// than SMs, whose stages in flight then are what hides the latency of a load
// (1003 x 1777 x 1000, 112 CTAs of 16 blocks: 12.0 us against 13.6).
template <int BN, bool DEEP>
struct Few {
    static constexpr int kStageBytes = 128 * kRowBytes + BN * kRowBytes;
    // two CTAs per SM, whose loads in flight together cover HBM's latency
    static constexpr int kStages = DEEP ? (200 * 1024) / kStageBytes : std::min(6, (110 * 1024) / kStageBytes);
    static constexpr int kRedBytes = BN * 128 * 4;
    static constexpr int kData = std::max(kStages * kStageBytes, kRedBytes);
    static constexpr int kSmem = 1024 + kData + 256;
};

template <int BN, bool E4M3, typename O, bool DEEP>
__global__ void __launch_bounds__(kFewThreads, 2)
linear_few_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                  const Epilogue e, const Axis axis, const unsigned int* skip, int seg_blocks, uint32_t tmem_cols,
                  unsigned int* status)
{
    using F = Few<BN, DEEP>;
    constexpr int NS = F::kStages;
    if (skip) {
        wait_for_previous();
        if (*skip != 0) return;
    }
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + F::kData);
    uint64_t* empty = full + NS;
    uint64_t* acc_full = empty + NS;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drained = acc_empty + 2;  // abort mode: every product issued has completed
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(drained + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_ptr + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int splits = gridDim.x;
    const int rank = blockIdx.x;  // the cluster spans x: the rank within it
    const int n0 = blockIdx.y * 128, m0 = blockIdx.z * BN;
    const int kb0 = (int)((long long)axis.blocks() * rank / splits);
    const int kb1 = (int)((long long)axis.blocks() * (rank + 1) / splits);
    const int count = kb1 - kb0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + i, 1);
            mbar_init(acc_empty + i, kFewWarps);
        }
        mbar_init(drained, 1);
        mbar_fence_init();
        *abort_flag = 0;
    }
    if (warp == kFewWarps + 1) {
        tmem_alloc(tmem_ptr, tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    if (threadIdx.x == 0) {
        // the weights' way from HBM begins while the kernel before this one ends (a
        // decode layer of one sequence, captured: 26.2 -> 25.3 us); if that one
        // writes them, L2 is where both meet
        int section = kb0 / axis.per, block = kb0 - section * axis.per;
        for (int i = 0; i < min(count, kPrefetch); ++i) {
            tma_prefetch_2d(&wmap, axis.w_col(section) + block * (E4M3 ? kRowBytes : kRowBytes / 2), n0);
            if (++block == axis.per) {
                block = 0;
                ++section;
            }
        }
        prefetch_tensormap(&xmap);
    }
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_ptr);
    wait_for_previous();
    let_next_begin();

    const int tokens = min(BN, e.M - m0);
    float* red = reinterpret_cast<float*>(sm);
    if (warp == kFewWarps) {
        if (elect_one_sync()) {
            int issued = 0, section = kb0 / axis.per, block = kb0 - section * axis.per;
            for (; issued < count; ++issued) {
                const int st = issued % NS;
                if (issued >= NS) wait_or_abort(empty + st, ((issued / NS) - 1) & 1, abort_flag, status);
                if (*abort_flag) break;
                uint8_t* a = sm + st * F::kStageBytes;
                const int k = block * (E4M3 ? kRowBytes : kRowBytes / 2);
                mbar_arrive_expect_tx(full + st, F::kStageBytes);
                tma_load_2d(a, &wmap, axis.w_col(section) + k, n0, full + st);
                tma_load_2d(a + 128 * kRowBytes, &xmap, axis.x_col(section) + k, m0, full + st);
                if (++block == axis.per) {
                    block = 0;
                    ++section;
                }
            }
            // loads in flight end before the CTA does (in abort mode the products
            // may not have waited for them)
            for (int i = max(0, issued - NS); i < issued; ++i)
                mbar_wait(full + i % NS, (i / NS) & 1, kPollLimit);
        }
    } else if (warp == kFewWarps + 1) {
        if (elect_one_sync()) {
            constexpr uint32_t idesc = E4M3 ? idesc_e4m3(128, BN) : idesc_bf16(128, BN, false, false);
            int unit = 0, r = 0;  // the segment and the block within it
            for (int i = 0; i < count; ++i) {
                const int st = i % NS, buf = unit & 1;
                if (r == 0 && unit >= 2) wait_or_abort(acc_empty + buf, ((unit >> 1) - 1) & 1, abort_flag, status);
                wait_or_abort(full + st, (i / NS) & 1, abort_flag, status);
                if (*abort_flag) break;
                tc_fence_after_sync();
                const uint32_t a = smem_addr(sm + st * F::kStageBytes);
                const uint64_t ad = sdesc_sw128(a, 16, 1024), bd = sdesc_sw128(a + 128 * kRowBytes, 16, 1024);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mma_step<E4M3, false>(tmem + (uint32_t)buf * BN, ad + 2 * j, bd + 2 * j, idesc, r != 0 || j != 0);
                mma_commit(empty + st);
                if (++r == seg_blocks || i == count - 1) {
                    mma_commit(acc_full + buf);
                    ++unit;
                    r = 0;
                }
            }
            if (*abort_flag) {
                mma_commit(drained);
                mbar_wait(drained, 0, kPollLimit);
            }
        }
    } else {
        // warps 0..3 and 4..7 take a lane quadrant (32 channels) each, every other
        // 16 tokens
        constexpr int kChunks = BN >= 32 ? BN / 32 : 1;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const int units = (count + seg_blocks - 1) / seg_blocks, c0 = (warp >> 2) * 16;
        float sum[kChunks * 16];
        for (int u = 0; u < units; ++u) {
            const int buf = u & 1;
            wait_or_abort(acc_full + buf, (u >> 1) & 1, abort_flag, status);
            tc_fence_after_sync();
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                if (c0 + 32 * i >= tokens) break;
                uint32_t v[16];
                tmem_ld16_sync(lanes + buf * BN + c0 + 32 * i, v);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    sum[16 * i + j] = u == 0 ? __uint_as_float(v[j]) : sum[16 * i + j] + __uint_as_float(v[j]);
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty + buf);
        }
        // into shared memory as [token][channel]: the last accumulator is full, so
        // every product has read its stages and their memory is free
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            if (c0 + 32 * i >= tokens) break;
#pragma unroll
            for (int j = 0; j < 16; ++j) red[(c0 + 32 * i + j) * 128 + (warp & 3) * 32 + lane] = sum[16 * i + j];
        }
    }
    __syncwarp();

    // this thread's four channels of every token it joins: neighbours where rows
    // of y and residual start on four elements, else a warp's width apart
    const bool vec = (e.N & 3) == 0;
    const int n = n0 + (vec ? lane * 4 : lane), step = vec ? 1 : 32;
    float ws[4], bias[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int nj = min(n + j * step, e.N - 1);
        ws[j] = E4M3 ? e.w_scale[nj] : 1.0f;
        bias[j] = e.bias ? e.bias[nj] : 0.0f;
    }
    if (splits > 1) cluster_sync();
    else __syncthreads();
    if (warp == kFewWarps + 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, tmem_cols);
    }
    const uint32_t red_addr = smem_addr(red);
    const O* res = static_cast<const O*>(e.residual);
    const int stride = kFewWarps * splits;  // tokens between a warp's
    // Joins PARTS parts (or fewer, in the order of the ranks) of TOKENS tokens: all
    // of their loads are under way before the first is used.
    auto join = [&](auto tokens_c, auto parts_c, int t0) {
        constexpr int TOKENS = decltype(tokens_c)::value, PARTS = decltype(parts_c)::value;
        float rs[TOKENS][4], sx[TOKENS], v[TOKENS][4];
        float4 p[TOKENS][PARTS];
#pragma unroll
        for (int i = 0; i < TOKENS; ++i) {
            const int t = min(t0 + i * stride, tokens - 1);  // past the last: that one again
            sx[i] = E4M3 ? e.x_scale[m0 + t] : 1.0f;
            if (res) {
                const O* from = res + (long long)(m0 + t) * e.N + n;
                Packed<O, 4> r;
                r.zero();
                if (vec && n < e.N) r.load(from);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    rs[i][j] = r.get(j);
                    if (!vec && n + j * step < e.N) rs[i][j] = static_cast<float>(from[j * step]);
                }
            }
            const uint32_t at = red_addr + (uint32_t)(t * 128 + (vec ? lane * 4 : lane)) * 4;
#pragma unroll
            for (int k = 0; k < PARTS; ++k) {
                if (k >= splits) break;
                const uint32_t from = PARTS > 1 ? map_rank(at, k) : at;
                if (vec) p[i][k] = ld_cluster_f4(from);
                else p[i][k] = make_float4(ld_cluster_f1(from), ld_cluster_f1(from + 128), ld_cluster_f1(from + 256),
                                           ld_cluster_f1(from + 384));
            }
        }
#pragma unroll
        for (int i = 0; i < TOKENS; ++i) {
            v[i][0] = p[i][0].x; v[i][1] = p[i][0].y; v[i][2] = p[i][0].z; v[i][3] = p[i][0].w;
#pragma unroll
            for (int k = 1; k < PARTS; ++k) {
                if (k >= splits) break;
                v[i][0] += p[i][k].x; v[i][1] += p[i][k].y; v[i][2] += p[i][k].z; v[i][3] += p[i][k].w;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (E4M3) v[i][j] = v[i][j] * sx[i] * ws[j];
                v[i][j] += bias[j];
            }
            if (e.act != SSD_ACT_NONE) {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = activate<O>(v[i][j], e.act);
            }
            if (res) {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] += rs[i][j];
            }
            const int t = t0 + i * stride;
            if (t >= tokens) break;
            O* y = static_cast<O*>(e.y) + (long long)(m0 + t) * e.N + n;
            if (vec) {
                Packed<O, 4> out;
                out.set(v[i]);
                if (n < e.N) out.store(y);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n + j * step < e.N) io<O>::store(y + j * step, v[i][j]);
            }
        }
    };
    int t = warp < kFewWarps ? rank + warp * splits : tokens;
    if (splits == 1) {
#pragma unroll 1
        for (; t < tokens; t += 4 * stride) join(Int<4>{}, Int<1>{}, t);
    } else if (splits == 2) {
#pragma unroll 1
        for (; t < tokens; t += 4 * stride) join(Int<4>{}, Int<2>{}, t);
    } else if (splits <= 4) {
#pragma unroll 1
        for (; t < tokens; t += 2 * stride) join(Int<2>{}, Int<4>{}, t);
    } else {
#pragma unroll 1
        for (; t < tokens; t += stride) join(Int<1>{}, Int<kMostSplits>{}, t);
    }
    if (splits > 1) cluster_sync();  // no CTA leaves while another reads its tile
}

template <int BN, bool E4M3, typename O, bool DEEP>
cudaError_t launch_few_as(const Operands& o, const Epilogue& e, int splits, const LaunchCtx& ctx)
{
    using F = Few<BN, DEEP>;
    const int es = E4M3 ? 1 : 2;
    const int kblocks = o.axis.blocks();
    const int tn = (e.N + 127) / 128, tm = (e.M + BN - 1) / BN;
    const int per = (kblocks + splits - 1) / splits;  // blocks of the longest part
    const int seg_blocks = sizeof(O) == 4 && !E4M3 ? kSegBlocks : per;
    const uint32_t cols = std::max(32, seg_blocks < per ? 2 * BN : BN);
    CUtensorMap wmap, xmap;
    if (!make_map_rows(&wmap, o.w, E4M3, o.w_cols, e.N, o.w_pitch * es, 128) ||
        !make_map_rows(&xmap, o.x, E4M3, o.x_cols, e.M, o.x_pitch * es, BN))
        return cudaErrorInvalidValue;
    auto* kernel = linear_few_kernel<BN, E4M3, O, DEEP>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t err = allow_smem(reinterpret_cast<const void*>(kernel), F::kSmem, allowed);
    if (err != cudaSuccess) return err;
    return launch_overlapped(kernel, dim3(splits, tn, tm), kFewThreads, F::kSmem, ctx.stream, splits, wmap, xmap, e, o.axis,
                             o.skip, seg_blocks, cols, ctx.status);
}

// ------------------------------------------------------------ many tokens

// A pair of CTAs computes 256 tokens x BN channels: each stages its own 128
// tokens and half of the channels, and one thread of the leader issues
// tcgen05.mma.cta_group::2 for both, so an operand byte is read from L2 and
// stored to shared memory once per pair instead of once per CTA. Accumulators
// (128 lanes = tokens, BN columns in each CTA) take turns in TMEM, so the
// epilogue of one runs under the products of the next.
//
// SEG (fp32 outputs of bf16 operands): the epilogue warps hold the tile in registers
// and join its segments there (see kSegBlocks).
template <int BN, bool SEG>
struct Many {
    static constexpr int kBRows = BN / 2;
    static constexpr int kStageBytes = (128 + kBRows) * kRowBytes;
    static constexpr int kStages = (196 * 1024) / kStageBytes;
    static constexpr int kBuffers = 512 / BN;
    // warps of a lane quadrant share its columns: with SEG each holds its 64 in
    // registers, without it 128 in passing
    static constexpr int kParts = SEG ? BN / 64 : 2;
    static constexpr int kEpiWarps = 4 * kParts;
    static constexpr int kThreads = 128 + 32 * kEpiWarps;
    // rows that do not start on 32 bytes leave through shared memory (see
    // store_staged): 32 tokens x kTurn channels to a warp
    static constexpr int kTurn = kEpiWarps > 8 ? 8 : 32;
    static constexpr int kTurnBytes = 32 * (kTurn + 1) * 4 * kEpiWarps;
    static constexpr int kSmem = 1024 + kStages * kStageBytes + kTurnBytes + 512;
    static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

// 32 bytes of one row (rows that allow it start on 32 bytes).
__device__ __forceinline__ void st32(void* p, const uint32_t* w)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
}
__device__ __forceinline__ void ld32(const void* p, uint32_t* w)
{
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p) : "memory");
}

// Four consecutive fp32 values that start on 16 bytes.
__device__ __forceinline__ void ld4(const float* p, float* v)
{
    const float4 f = *reinterpret_cast<const float4*>(p);
    v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
}

// The epilogue of CH channels from n (a multiple of CH, all of them within the
// row) of token m, rows that start on 32 bytes: the thread's accumulators to y.
template <int CH, bool E4M3, typename O>
__device__ __forceinline__ void store_row(const Epilogue& e, const void* residual, float* v, int m, int n, float sx)
{
    const long long at = (long long)m * e.N + n;
    O* y = static_cast<O*>(e.y) + at;
    const O* res = static_cast<const O*>(residual);
    constexpr int kWords = CH * (int)sizeof(O) / 4;
    uint32_t r[kWords];
    if (res) {
#pragma unroll
        for (int i = 0; i < kWords; i += 8) ld32(res + at + i * 4 / (int)sizeof(O), r + i);
    }
#pragma unroll
    for (int c = 0; c < CH; c += 4) {
        float b[4];
        if constexpr (E4M3) {
            ld4(e.w_scale + n + c, b);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[c + j] = v[c + j] * sx * b[j];
        }
        if (e.bias) {
            ld4(e.bias + n + c, b);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[c + j] += b[j];
        }
    }
    if (e.act == SSD_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < CH; ++j) v[j] = silu_f<O>(v[j]);
    } else if (e.act == SSD_ACT_GELU) {
        // rolled for the sake of the code's length; rotating the values by 8 keeps
        // their indexes constants
#pragma unroll 1
        for (int c = 0; c < CH; c += 8) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float t = gelu_f<O>(v[j]);
#pragma unroll
                for (int i = j; i + 8 < CH; i += 8) v[i] = v[i + 8];
                v[CH - 8 + j] = t;
            }
        }
    }
    Packed<O, CH> p;
    if (res) {
        Packed<O, CH> q;
#pragma unroll
        for (int i = 0; i < kWords; ++i) q.w[i] = r[i];
#pragma unroll
        for (int j = 0; j < CH; ++j) v[j] += q.get(j);
    }
    p.set(v);
#pragma unroll
    for (int i = 0; i < kWords; i += 8) st32(y + i * 4 / (int)sizeof(O), p.w + i);
}

// The same for rows of any alignment, and for the last channels of a row: the
// warp turns 32 tokens x CH channels round in shared memory (rows of CH + 1: no
// bank conflicts), so that its lanes take neighbouring channels and every access
// to y and residual is one run of a row. Called by the whole warp; m: the lane's
// own token.
template <int CH, bool E4M3, typename O>
__device__ __forceinline__ void store_staged(const Epilogue& e, const void* residual, const float* v, float* turn, int m,
                                             int n, float sx)
{
    const int lane = threadIdx.x & 31, m0 = m - lane;
    constexpr int kRowsAtOnce = 32 / CH;  // of a row of CH channels
    __syncwarp();
#pragma unroll
    for (int j = 0; j < CH; ++j) turn[lane * (CH + 1) + j] = v[j];
    __syncwarp();
    const int c = lane % CH, nc = n + c;
    const float ws = E4M3 ? e.w_scale[min(nc, e.N - 1)] : 1.0f;
    const float bias = e.bias ? e.bias[min(nc, e.N - 1)] : 0.0f;
    constexpr int kBatch = 8 < CH ? 8 : CH;  // rows under way together
    const int first = lane / CH;
    const int rows = nc < e.N ? min(32, e.M - m0) : 0;  // those of this lane's channel
    const long long at = (long long)(m0 + first) * e.N + nc, step = (long long)kRowsAtOnce * e.N;
    const O* res = residual ? static_cast<const O*>(residual) + at : nullptr;
    O* y = static_cast<O*>(e.y) + at;
#pragma unroll 1
    for (int r0 = first; r0 < 32; r0 += kRowsAtOnce * kBatch) {
        float rs[kBatch], f[kBatch];
        if (res) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i, res += step)
                rs[i] = r0 + i * kRowsAtOnce < rows ? static_cast<float>(*res) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = r0 + i * kRowsAtOnce;
            f[i] = turn[r * (CH + 1) + c];
            if constexpr (E4M3) f[i] = f[i] * __shfl_sync(0xffffffffu, sx, r) * ws;
            f[i] += bias;
        }
        if (e.act != SSD_ACT_NONE) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) f[i] = activate<O>(f[i], e.act);
        }
        if (res) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) f[i] += rs[i];
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i, y += step)
            if (r0 + i * kRowsAtOnce < rows) io<O>::store(y, f[i]);
    }
}

struct Tiles {
    int tm, tn;    // tiles along the tokens and the channels
    int group;     // tile rows walked together
    long long all;
};

// Tiles in groups of `group` rows, column by column within a group, so that the
// tiles in flight at once share operands in L2.
__device__ __forceinline__ void tile_at(const Tiles& t, long long i, int& im, int& in)
{
    const long long per = (long long)t.group * t.tn;
    const int g = (int)(i / per);
    const int rows = min(t.group, t.tm - g * t.group);
    const int r = (int)(i - g * per);
    im = g * t.group + r % rows;
    in = r / rows;
}

template <int BN, bool E4M3, typename O, bool SEG, bool WIDE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Many<BN, SEG>::kThreads, 1)
linear_many_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                   const Epilogue e, const Tiles tiles, const Axis axis, const unsigned int* skip, unsigned int* status)
{
    using T = Many<BN, SEG>;
    constexpr int NS = T::kStages, NB = T::kBuffers;
    if (skip) {
        wait_for_previous();
        if (*skip != 0) return;
    }
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + NS * T::kStageBytes + T::kTurnBytes);  // leader's: both CTAs' loads
    uint64_t* empty = full + NS;          // each CTA's
    uint64_t* acc_full = empty + NS;      // each CTA's
    uint64_t* acc_empty = acc_full + NB;  // leader's: both CTAs' epilogue warps
    uint64_t* drained = acc_empty + NB;   // each CTA's: every product issued has completed
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(drained + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_ptr + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int kblocks = axis.blocks();
    const int seg = SEG ? kSegBlocks : kblocks;  // K blocks of one accumulator
    const int segs = SEG ? (kblocks + seg - 1) / seg : 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < NB; ++i) {
            mbar_init(acc_full + i, 1);
            mbar_init(acc_empty + i, 2 * T::kEpiWarps);
        }
        mbar_init(drained, 1);
        mbar_fence_init();
        *abort_flag = 0;
    }
    if (warp == 2) tmem_alloc_pair(tmem_ptr, 512);
    tc_fence_before_sync();
    __syncthreads();
    if (threadIdx.x == 32) {
        prefetch_tensormap(&wmap);
        prefetch_tensormap(&xmap);
    }
    cluster_sync();  // barriers of both CTAs are set up
    tc_fence_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_ptr);
    wait_for_previous();
    let_next_begin();

    if (warp == 0) {
        if (elect_one_sync()) {
            long long it = 0;
            for (long long i = pair; i < tiles.all && !*abort_flag; i += pairs) {
                int im, in;
                tile_at(tiles, i, im, in);
                const int m = im * 256 + (int)rank * 128, n = in * BN + (int)rank * T::kBRows;
                int section = 0, block = 0;
                for (int kb = 0; kb < kblocks; ++kb, ++it) {
                    const int st = (int)(it % NS);
                    if (it >= NS) wait_or_abort(empty + st, (uint32_t)((it / NS) - 1) & 1, abort_flag, status);
                    if (*abort_flag) break;
                    uint8_t* a = sm + st * T::kStageBytes;
                    const int k = block * (E4M3 ? kRowBytes : kRowBytes / 2);
                    // the leader's barrier counts both CTAs' bytes
                    if (rank == 0) mbar_arrive_expect_tx(full + st, 2 * T::kStageBytes);
                    const uint32_t bar = map_rank(smem_addr(full + st), 0);
                    tma_load_2d_pair(a, &xmap, axis.x_col(section) + k, m, bar);
                    tma_load_2d_pair(a + 128 * kRowBytes, &wmap, axis.w_col(section) + k, n, bar);
                    if (++block == axis.per) {
                        block = 0;
                        ++section;
                    }
                }
            }
            // every stage loaded has been read by the MMAs: none is in flight when
            // the CTA ends, nor a commit's arrival on this CTA's barriers
            for (long long j = it > NS ? it - NS : 0; j < it; ++j)
                mbar_wait(empty + j % NS, (uint32_t)(j / NS) & 1, kPollLimit);
        }
    } else if (warp == 1 && rank != 0) {
        if (elect_one_sync()) wait_or_abort(drained, 0, abort_flag, status);
    } else if (warp == 1) {
        if (elect_one_sync()) {
            constexpr uint32_t idesc = E4M3 ? idesc_e4m3(256, BN) : idesc_bf16(256, BN, false, false);
            long long it = 0, unit = 0;
            for (long long i = pair; i < tiles.all && !*abort_flag; i += pairs) {
                for (int kb = 0; kb < kblocks; ++kb, ++it) {
                    const int buf = (int)(unit % NB);
                    const bool first = kb % seg == 0;
                    if (first) {
                        if (unit >= NB)
                            wait_or_abort(acc_empty + buf, (uint32_t)((unit / NB) - 1) & 1, abort_flag, status);
                        tc_fence_after_sync();
                    }
                    const int st = (int)(it % NS);
                    wait_or_abort(full + st, (uint32_t)(it / NS) & 1, abort_flag, status);
                    if (*abort_flag) break;
                    tc_fence_after_sync();
                    const uint32_t a = smem_addr(sm + st * T::kStageBytes);
                    const uint64_t ad = sdesc_sw128(a, 16, 1024), bd = sdesc_sw128(a + 128 * kRowBytes, 16, 1024);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_step<E4M3, true>(tmem + buf * BN, ad + 2 * j, bd + 2 * j, idesc, !first || j != 0);
                    mma_commit_pair(empty + st);
                    if (kb % seg == seg - 1 || kb == kblocks - 1) {
                        mma_commit_pair(acc_full + buf);
                        ++unit;
                    }
                }
            }
            mma_commit_pair(drained);
            mbar_wait(drained, 0, kPollLimit);
        }
    } else if (warp >= 4) {
        // each quadrant of 32 lanes belongs to the warps of its number mod 4
        const int quad = warp & 3, part = (warp - 4) >> 2;
        constexpr int kCols = BN / T::kParts;
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16) + part * kCols;
        float* turn = reinterpret_cast<float*>(sm + NS * T::kStageBytes) + (warp - 4) * 32 * (T::kTurn + 1);
        long long unit = 0;
        for (long long i = pair; i < tiles.all && !*abort_flag; i += pairs) {
            int im, in;
            tile_at(tiles, i, im, in);
            const int m = im * 256 + (int)rank * 128 + quad * 32 + lane;
            const int n = in * BN + part * kCols;
            const float sx = E4M3 && m < e.M ? e.x_scale[m] : 1.0f;
            float sum[SEG ? kCols : 1];
            // without an activation the sum may begin with the residual, which is
            // then read while the first products are under way
            const bool early = SEG && WIDE && e.residual && e.act == SSD_ACT_NONE && n + kCols <= e.N;
            if constexpr (SEG) {
#pragma unroll
                for (int c = 0; c < kCols; ++c) sum[c] = 0.0f;
                if constexpr (WIDE) {
                    if (early && m < e.M) {
                        const O* res = static_cast<const O*>(e.residual) + (long long)m * e.N + n;
#pragma unroll
                        for (int c = 0; c < kCols; c += 8) ld32(res + c, reinterpret_cast<uint32_t*>(sum) + c);
                    }
                }
            }
            for (int s = 0; s < segs; ++s, ++unit) {
                const int buf = (int)(unit % NB);
                wait_or_abort(acc_full + buf, (uint32_t)(unit / NB) & 1, abort_flag, status);
                tc_fence_after_sync();
                if constexpr (SEG) {
#pragma unroll
                    for (int c = 0; c < kCols; c += 16) {
                        uint32_t v[16];
                        tmem_ld16_sync(lanes + buf * BN + c, v);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            sum[c + j] += __uint_as_float(v[j]);
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < kCols; c += 32) {
                        uint32_t v[32];
                        tmem_ld32_sync(lanes + buf * BN + c, v);
                        float f[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(v[j]);
                        if (*abort_flag) continue;
                        if (WIDE && n + c + 32 <= e.N) {
                            if (m < e.M) store_row<32, E4M3, O>(e, e.residual, f, m, n + c, sx);
                        } else if (n + c < e.N) {
                            store_staged<32, E4M3, O>(e, e.residual, f, turn, m, n + c, sx);
                        }
                    }
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_rank(smem_addr(acc_empty + buf), 0));
            }
            if constexpr (SEG) {
                const void* residual = early ? nullptr : e.residual;
                if (*abort_flag) continue;
                if (WIDE && n + kCols <= e.N) {
                    if (m < e.M) {
#pragma unroll
                        for (int c = 0; c < kCols; c += 8) store_row<8, E4M3, O>(e, residual, sum + c, m, n + c, sx);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < kCols; c += T::kTurn)
                        if (n + c < e.N) store_staged<T::kTurn, E4M3, O>(e, residual, sum + c, turn, m, n + c, sx);
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    // all of the pair's products have been read and all arrivals on its barriers
    // have landed before either CTA ends
    cluster_sync();
    tc_fence_after_sync();
    if (warp == 2) tmem_dealloc_pair(tmem, 512);
}

// Whether rows of y and residual start on 32 bytes.
template <typename O>
bool wide_rows(const Epilogue& e)
{
    return (long long)e.N * sizeof(O) % 32 == 0 && aligned_to(e.y, 32) && aligned_to(e.residual, 32);
}

template <int BN, bool E4M3, typename O, bool SEG>
cudaError_t launch_many(const Operands& o, const Epilogue& e, const LaunchCtx& ctx)
{
    using T = Many<BN, SEG>;
    const int es = E4M3 ? 1 : 2;
    Tiles t;
    t.tm = (int)(((long long)e.M + 255) / 256);
    t.tn = (e.N + BN - 1) / BN;
    t.group = 8;
    t.all = (long long)t.tm * t.tn;
    CUtensorMap wmap, xmap;
    if (!make_map_rows(&wmap, o.w, E4M3, o.w_cols, e.N, o.w_pitch * es, T::kBRows) ||
        !make_map_rows(&xmap, o.x, E4M3, o.x_cols, e.M, o.x_pitch * es, 128))
        return cudaErrorInvalidValue;
    auto* kernel = linear_many_kernel<BN, E4M3, O, SEG, true>;
    if constexpr (!(SEG && BN == 256)) {
        if (!wide_rows<O>(e)) kernel = linear_many_kernel<BN, E4M3, O, SEG, false>;
    }
    static std::atomic<uint64_t> allowed[2];
    cudaError_t err = allow_smem(reinterpret_cast<const void*>(kernel), T::kSmem, allowed[wide_rows<O>(e)]);
    if (err != cudaSuccess) return err;
    const int pairs = (int)std::min<long long>(t.all, ctx.num_sms / 2);
    // the kernel's own attribute makes the pairs clusters of two
    return launch_overlapped(kernel, 2 * pairs, T::kThreads, T::kSmem, ctx.stream, 1, wmap, xmap, e, t, o.axis, o.skip,
                             ctx.status);
}

// ------------------------------------------------------------------ choice

// How many clusters of `splits` CTAs of the few-token kernel the device holds at
// once (a GPC takes whole clusters only: 90, 44 and 30 of 3, 6 and 8 here); asks
// the runtime once. Its answer counts one CTA per SM, of two.
template <int BN, bool E4M3, typename O>
int active_clusters(int splits, int num_sms)
{
    static std::atomic<int> known[64][kMostSplits + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return num_sms / splits;
    int n = known[dev & 63][splits].load(std::memory_order_relaxed);
    if (n) return n;
    using F = Few<BN, false>;
    auto* kernel = linear_few_kernel<BN, E4M3, O, false>;
    static std::atomic<uint64_t> allowed{0};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(splits, 1024);
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = F::kSmem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = splits;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (allow_smem(reinterpret_cast<const void*>(kernel), F::kSmem, allowed) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = std::max(1, num_sms / splits);
    }
    if (n * splits <= num_sms) n *= 2;
    known[dev & 63][splits].store(n, std::memory_order_relaxed);
    return n;
}

template <int BN, bool E4M3, typename O>
cudaError_t launch_few(const Operands& o, const Epilogue& e, int splits, const LaunchCtx& ctx)
{
    if constexpr (BN >= 64) {
        const long long tiles = (long long)((e.N + 127) / 128) * ((e.M + BN - 1) / BN);
        const int room = splits == 1 ? ctx.num_sms : active_clusters<BN, E4M3, O>(splits, ctx.num_sms) / 2;
        if (tiles <= room && (o.axis.blocks() + splits - 1) / splits > Few<BN, false>::kStages)
            return launch_few_as<BN, E4M3, O, true>(o, e, splits, ctx);
    }
    return launch_few_as<BN, E4M3, O, false>(o, e, splits, ctx);
}

int tokens_per_tile(int M) { return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128; }

// Estimated microseconds of a call, fitted to measurements of both kernels over
// 1 to 2048 tokens and five weight shapes from 1024 x 2048 to 10576 x 2560, bf16
// and e4m3 (off by a tenth on most, by a quarter at worst). A pair's tile takes
// 0.31 us a block of K at 256 channels, where tensor cores and L2 balance, and
// 0.215 at 128, where L2 bounds it; 2.5 and 1.5 us for its ends, and 2 more where
// its rows leave through shared memory. The few-token
// kernel takes 3.4 to 4.7 us for its ends with the tokens, 0.5 to 2 more where parts
// of K are joined, and the largest of its chain of stages (0.28 us a block), its
// traffic from L2 at 15 TB/s and the weights from HBM at 6 TB/s, with some of the
// other two.
float many_us(long long tm, int N, int BN, int kblocks, bool wide, int num_sms)
{
    const long long tiles = tm * ((N + BN - 1) / BN), pairs = num_sms / 2;
    const float waves = (float)((tiles + pairs - 1) / pairs);
    return 5.0f + waves * ((BN == 256 ? 0.31f * kblocks + 2.5f : 0.215f * kblocks + 1.5f) + (wide ? 0.0f : 2.0f));
}
float few_us(int BN, long long tiles, int N, int kblocks, int splits, int num_sms)
{
    const float waves = (float)((tiles * splits + 2ll * num_sms - 1) / (2ll * num_sms));
    const float chain = waves * 0.28f * ((kblocks + splits - 1) / splits);
    const float traffic = (float)tiles * kblocks * (128 + BN) * kRowBytes / 15e6f;
    const float weights = (float)N * kblocks * kRowBytes / 6e6f;
    const float ends = 3.2f + 0.012f * BN + (splits > 1 ? 0.3f + 0.012f * BN + 0.1f * splits : 0.0f);
    const float longest = std::max(chain, std::max(traffic, weights));
    return waves * ends + 0.85f * longest + 0.15f * (chain + traffic + weights);
}

// The parts of K of a call of the few-token kernel: the fewest of the shortest
// estimate among those whose clusters all run at once, two blocks to a part.
template <int BN, bool E4M3, typename O>
int few_splits(long long tiles, int N, int kblocks, int num_sms)
{
    int best = 1;
    for (int s = 2; s <= std::min(kMostSplits, kblocks / 2); ++s) {
        if (tiles * s > 2ll * num_sms || tiles > active_clusters<BN, E4M3, O>(s, num_sms)) break;
        if (few_us(BN, tiles, N, kblocks, s, num_sms) < few_us(BN, tiles, N, kblocks, best, num_sms)) best = s;
    }
    return best;
}

template <bool E4M3, typename O>
int splits_for(int BN, long long tiles, int N, int kblocks, int num_sms)
{
    switch (BN) {
    case 16: return few_splits<16, E4M3, O>(tiles, N, kblocks, num_sms);
    case 32: return few_splits<32, E4M3, O>(tiles, N, kblocks, num_sms);
    case 64: return few_splits<64, E4M3, O>(tiles, N, kblocks, num_sms);
    default: return few_splits<128, E4M3, O>(tiles, N, kblocks, num_sms);
    }
}

template <bool E4M3, typename O>
cudaError_t run(const Operands& o, const Epilogue& e, const LaunchCtx& ctx)
{
    constexpr bool kSeg = sizeof(O) == 4 && !E4M3;
    const int kblocks = o.axis.blocks(), BN = tokens_per_tile(e.M), sms = ctx.num_sms, variant = g_variant;
    const long long tiles = (long long)((e.N + 127) / 128) * ((e.M + BN - 1) / BN), tm = ((long long)e.M + 255) / 256;
    const bool wide = wide_rows<O>(e);
    const float many256 = many_us(tm, e.N, 256, kblocks, wide, sms);
    const float many128 = many_us(tm, e.N, 128, kblocks, wide, sms);
    const bool fits = (e.M + BN - 1) / BN <= 65535;  // the grid's z extent
    if (variant != 3 && fits) {
        const int splits = splits_for<E4M3, O>(BN, tiles, e.N, kblocks, sms);
        if (variant == 2 || few_us(BN, tiles, e.N, kblocks, splits, sms) <= std::min(many256, many128)) {
            switch (BN) {
            case 16: return launch_few<16, E4M3, O>(o, e, splits, ctx);
            case 32: return launch_few<32, E4M3, O>(o, e, splits, ctx);
            case 64: return launch_few<64, E4M3, O>(o, e, splits, ctx);
            default: return launch_few<128, E4M3, O>(o, e, splits, ctx);
            }
        }
    }
    // sixteen warps that turn rows round have room for 8 channels at a time, 32 bytes
    // of a row; the eight of the narrower tile for 32 (16384 x 10001 x 1024: 668 us
    // against 454)
    return many128 < many256 || (kSeg && !wide) ? launch_many<128, E4M3, O, kSeg>(o, e, ctx) : launch_many<256, E4M3, O, kSeg>(o, e, ctx);
}

int element_bytes(const LinearArgs& a) { return a.type == LinearType::e4m3 ? 1 : a.type == LinearType::bf16 ? 2 : 4; }
long long round_up(long long v, long long m) { return (v + m - 1) / m * m; }

// TMA addresses rows of 16-byte multiples from 16-byte bases.
bool x_addressable(const LinearArgs& a)
{
    return aligned_to(a.x, 16) && a.x_stride * element_bytes(a) % 16 == 0;
}
bool w_addressable(const LinearArgs& a) { return (long long)a.K * element_bytes(a) % 16 == 0; }

// How a call's operands reach the kernels.
enum class Path { direct, pack, split, rows, simt };

// Operands that the tensor cores take as they lie go there. The others pay for
// another copy of the weights, or, for a few tokens, are read as they lie by the rows
// kernel: whichever takes less by these estimates, fitted to 1 to 32 tokens of 300 x
// 700 to 10576 x 2561 (microseconds; the copies' own launches are their constants).
Path path_of(const LinearArgs& a)
{
    if (g_variant == 1) return Path::simt;
    const bool f32 = a.type == LinearType::f32, addressable = x_addressable(a) && w_addressable(a);
    if (!f32 && addressable) return Path::direct;
    const float nk = 1e-6f * a.N * a.K;
    const float each = addressable || (a.type == LinearType::e4m3 && a.M == 1) ? 0.65f : 1.4f;
    const float rows = 2.0f + nk * std::max(each, 0.27f * a.M);
    const float copies = f32 ? 12.0f + 3.5f * nk : 8.0f + 1.15f * nk;
    if (g_variant == 0 && a.M <= (f32 ? 32 : 16) && rows <= copies) return Path::rows;
    return f32 ? Path::split : Path::pack;
}

// Workspace: a flag (256 bytes), then x's copy, then w's.
struct Copies {
    long long x_pitch, w_pitch, cols;  // elements; cols: of one section
    size_t x_at, w_at, bytes;
};
Copies copies_of(const LinearArgs& a, Path path)
{
    Copies c = {};
    const int es = path == Path::split ? 2 : element_bytes(a), sections = path == Path::split ? 3 : 1;
    c.cols = round_up(a.K, kRowBytes / es);
    c.x_pitch = c.w_pitch = c.cols * sections;
    c.x_at = 256;
    const bool copy_x = path == Path::split || !x_addressable(a), copy_w = path == Path::split || !w_addressable(a);
    c.w_at = c.x_at + (copy_x ? (size_t)round_up((long long)a.M * c.x_pitch * es, 256) : 0);
    c.bytes = c.w_at + (copy_w ? (size_t)round_up((long long)a.N * c.w_pitch * es, 256) : 0);
    return c;
}

template <bool E4M3>
cudaError_t run_out(const Operands& o, const Epilogue& e, bool out_bf16, const LaunchCtx& ctx)
{
    return out_bf16 ? run<E4M3, __nv_bfloat16>(o, e, ctx) : run<E4M3, float>(o, e, ctx);
}

// fp32 operands on the bf16 tensor cores: x = x1 + x2 + x3 and w = w1 + w2 + w3
// with 8 significant bits each, so
//     x w = x1 w1 + (x1 w2 + x2 w1) + (x1 w3 + x2 w2 + x3 w1) + O(2^-24),
// one product over six sections of K (a sixth of the tensor cores' bf16 rate against the
// SIMT kernel's 19 TFLOP/s). Products of infinities do not split: when a value of the
// operands does not fit bf16's range, at its top or with its last bits at its bottom,
// the tensor-core kernel stands back and the SIMT kernel computes the call (64 x 10576 x
// 2560 393 us instead of 114, 16384 x 10576 x 2560 43 ms instead of 3.7).
cudaError_t linear_split(const LinearArgs& a, const Epilogue& e, char* ws, const LaunchCtx& ctx)
{
    const Copies c = copies_of(a, Path::split);
    unsigned int* flag = reinterpret_cast<unsigned int*>(ws);
    cudaError_t err = cudaMemsetAsync(flag, 0, sizeof(*flag), ctx.stream);
    if (err == cudaSuccess)
        err = split_rows(static_cast<const float*>(a.x), a.x_stride, a.M, a.K, ws + c.x_at, (int)c.cols, flag, ctx);
    if (err == cudaSuccess)
        err = split_rows(static_cast<const float*>(a.w), a.K, a.N, a.K, ws + c.w_at, (int)c.cols, flag, ctx);
    if (err != cudaSuccess) return err;
    Operands o;
    o.x = ws + c.x_at;
    o.w = ws + c.w_at;
    o.x_cols = o.x_pitch = o.w_cols = o.w_pitch = c.x_pitch;
    // sections (x, w): (3, 1), (2, 2), (1, 3), (2, 1), (1, 2), (1, 1)
    o.axis = {(int)(c.cols / (kRowBytes / 2)), 6, (int)c.cols,
              2u | 1u << 2 | 0u << 4 | 1u << 6 | 0u << 8 | 0u << 10,
              0u | 1u << 2 | 2u << 4 | 0u << 6 | 1u << 8 | 0u << 10};
    o.skip = flag;
    err = run_out<false>(o, e, a.out_bf16, ctx);
    return err == cudaSuccess ? linear_simt(a, flag, ctx) : err;
}

}  // namespace

void set_linear_variant(int variant) { g_variant = variant >= 0 && variant <= 3 ? variant : 0; }

size_t linear_workspace_bytes(const LinearArgs& a)
{
    const Path path = path_of(a);
    return path == Path::pack || path == Path::split ? copies_of(a, path).bytes : 0;
}

cudaError_t linear(const LinearArgs& a, void* workspace, const LaunchCtx& ctx)
{
    const Path path = path_of(a);
    const Epilogue e{a.x_scale, a.w_scale, a.bias, a.residual, a.y, a.M, a.N, a.act};
    char* ws = static_cast<char*>(workspace);
    if (path == Path::simt) return linear_simt(a, nullptr, ctx);
    if (path == Path::rows) return linear_rows(a, ctx);
    if (path == Path::split) return linear_split(a, e, ws, ctx);
    Operands o;
    o.x = a.x;
    o.w = a.w;
    o.x_pitch = a.x_stride;
    o.w_pitch = a.K;
    o.x_cols = o.w_cols = a.K;
    if (path == Path::pack) {
        const Copies c = copies_of(a, path);
        cudaError_t err = cudaSuccess;
        if (!x_addressable(a)) {
            o.x = ws + c.x_at;
            o.x_pitch = c.x_pitch;
            err = pack_rows(a.x, a.x_stride, a.M, a.K, a.type, ws + c.x_at, (int)c.x_pitch, ctx);
        }
        if (err == cudaSuccess && !w_addressable(a)) {
            o.w = ws + c.w_at;
            o.w_pitch = c.w_pitch;
            err = pack_rows(a.w, a.K, a.N, a.K, a.type, ws + c.w_at, (int)c.w_pitch, ctx);
        }
        if (err != cudaSuccess) return err;
    }
    const int unit = kRowBytes / element_bytes(a);
    o.axis = {(a.K + unit - 1) / unit, 1, 0, 0u, 0u};
    o.skip = nullptr;
    return a.type == LinearType::e4m3 ? run_out<true>(o, e, a.out_bf16, ctx) : run_out<false>(o, e, a.out_bf16, ctx);
}

}  // namespace ssd
