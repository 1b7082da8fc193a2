// norm.cu -- layer norm forward (with the residual add) and backward (with the
// reduction of the weight's and bias's gradients).
//
//   S = X + R (rounded to the stored type)     mu = mean(S), r = 1 / sqrt(mean((S - mu)^2) + eps)
//   Y = (S - mu) r gamma + beta                xh = (S - mu) r,  g = dY gamma
//   dX = r (g - mean(g) - xh mean(g xh)) + dS  dgamma = sum_t dY xh,  dbeta = sum_t dY
//
// Both directions are bound by HBM: each tensor crosses it once.  All sums are
// fp32, in a fixed order (no atomics), so results repeat bit for bit.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "train.h"

namespace tffn {
namespace norm {

// A vector of VW activations as it lies in memory.
template <typename T, int VW>
struct alignas(sizeof(T) * VW) Vec {
    T e[VW];
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v)
{
    return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v)
{
    return __float2bfloat16_rn(v);
}

// Words of 16, 8, 4 or 2 bytes.
template <int B>
struct Word;
template <>
struct Word<16> { using type = uint4; };
template <>
struct Word<8> { using type = uint2; };
template <>
struct Word<4> { using type = uint32_t; };
template <>
struct Word<2> { using type = uint16_t; };

// Streaming load and store: the tensors are read and written once.
template <typename T, int VW>
__device__ __forceinline__ Vec<T, VW> load_stream(const T* p)
{
    using W = typename Word<sizeof(T) * VW>::type;
    const W w = __ldcs(reinterpret_cast<const W*>(p));
    return *reinterpret_cast<const Vec<T, VW>*>(&w);
}

template <typename T, int VW>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, VW>& v)
{
    using W = typename Word<sizeof(T) * VW>::type;
    *reinterpret_cast<W*>(p) = *reinterpret_cast<const W*>(&v);
}

// VW parameters from column c; `absent` where there is no tensor.
template <int VW>
__device__ __forceinline__ void load_param(const void* p, bool f32, int64_t c, float absent, bool vec, float (&v)[VW])
{
    if (p == nullptr) {
#pragma unroll
        for (int j = 0; j < VW; ++j)
            v[j] = absent;
    } else if (f32) {
        const float* q = static_cast<const float*>(p) + c;
        if (VW % 4 == 0 && vec) {
#pragma unroll
            for (int j = 0; j < VW / 4; ++j) {
                const float4 x = __ldg(reinterpret_cast<const float4*>(q) + j);
                v[4 * j] = x.x;
                v[4 * j + 1] = x.y;
                v[4 * j + 2] = x.z;
                v[4 * j + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < VW; ++j)
                v[j] = __ldg(q + j);
        }
    } else {
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p) + c;
        if (VW % 4 == 0 && vec) {
#pragma unroll
            for (int j = 0; j < VW / 4; ++j) {
                const uint2 x = __ldg(reinterpret_cast<const uint2*>(q) + j);
                v[4 * j] = __uint_as_float(x.x << 16);
                v[4 * j + 1] = __uint_as_float(x.x & 0xFFFF0000u);
                v[4 * j + 2] = __uint_as_float(x.y << 16);
                v[4 * j + 3] = __uint_as_float(x.y & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < VW; ++j)
                v[j] = __bfloat162float(q[j]);
        }
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the TPR threads of a row (a warp, or the whole block).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red)
{
    v = warp_sum(v);
    if (TPR == 32)
        return v;
    constexpr int NW = TPR / 32;
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NW; ++i)
        s += red[i];
    return s;
}

struct FwdArgs {
    const void *X, *R, *gamma, *beta;
    void *Y, *S;
    float *mean, *rstd;
    int64_t T, N;
    float eps;
    int p32, pvec;
};

// A row's columns stay in the registers of its TPR threads (NV vectors of VW
// each), so the row is read once and the variance is the exact second pass
// over (S - mu).  Rows of up to 512 bytes a thread's warp owns; longer rows
// take a block.
template <typename T, int VW, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) norm_fwd_kernel(const FwdArgs a)
{
    __shared__ float red[2][TPR <= 32 ? 1 : TPR / 32];
    constexpr int ROWS = TPR < 128 ? 128 / TPR : 1;   // rows per block
    const int t = threadIdx.x % TPR;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / TPR;
    if (row >= a.T)
        return;   // whole warps: a block with several warps per row holds one row
    const T* x = static_cast<const T*>(a.X) + row * a.N;
    const T* r = a.R == nullptr ? nullptr : static_cast<const T*>(a.R) + row * a.N;
    Vec<T, VW> xv[NV], rv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = static_cast<int64_t>(i * TPR + t) * VW;
        if (c < a.N) {
            xv[i] = load_stream<T, VW>(x + c);
            if (r != nullptr)
                rv[i] = load_stream<T, VW>(r + c);
        }
    }
    float v[NV][VW];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = static_cast<int64_t>(i * TPR + t) * VW;
#pragma unroll
        for (int j = 0; j < VW; ++j)
            v[i][j] = 0.0f;
        if (c < a.N) {
            if (r != nullptr) {
                // the norm is of S as it is stored
#pragma unroll
                for (int j = 0; j < VW; ++j)
                    xv[i].e[j] = from_f<T>(to_f(xv[i].e[j]) + to_f(rv[i].e[j]));
                store_vec<T, VW>(static_cast<T*>(a.S) + row * a.N + c, xv[i]);
            }
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                v[i][j] = to_f(xv[i].e[j]);
                sum += v[i][j];
            }
        }
    }
    const float inv_n = 1.0f / static_cast<float>(a.N);
    const float mean = row_sum<TPR>(sum, red[0]) * inv_n;
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = static_cast<int64_t>(i * TPR + t) * VW;
        if (c < a.N) {
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                const float d = v[i][j] - mean;
                sq = fmaf(d, d, sq);
            }
        }
    }
    const float rstd = rsqrtf(row_sum<TPR>(sq, red[1]) * inv_n + a.eps);
    if (t == 0) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = static_cast<int64_t>(i * TPR + t) * VW;
        if (c < a.N) {
            float g[VW], b[VW];
            load_param<VW>(a.gamma, a.p32, c, 1.0f, a.pvec, g);
            load_param<VW>(a.beta, a.p32, c, 0.0f, a.pvec, b);
            Vec<T, VW> y;
#pragma unroll
            for (int j = 0; j < VW; ++j)
                y.e[j] = from_f<T>(fmaf((v[i][j] - mean) * rstd, g[j], b[j]));
            store_vec<T, VW>(static_cast<T*>(a.Y) + row * a.N + c, y);
        }
    }
}

// Rows too long for registers: one block per row, three passes over the row
// (the second and third mostly from L2).
template <typename T>
__global__ void __launch_bounds__(1024) norm_fwd_long_kernel(const FwdArgs a)
{
    __shared__ float red[2][32];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.X) + row * a.N;
    const T* r = a.R == nullptr ? nullptr : static_cast<const T*>(a.R) + row * a.N;
    T* s = static_cast<T*>(a.S) + row * a.N;
    float sum = 0.0f;
    for (int64_t c = threadIdx.x; c < a.N; c += 1024) {
        T v = x[c];
        if (r != nullptr) {
            v = from_f<T>(to_f(v) + to_f(r[c]));
            s[c] = v;
        }
        sum += to_f(v);
    }
    const T* in = r != nullptr ? s : x;   // each thread reads back what it wrote itself
    const float inv_n = 1.0f / static_cast<float>(a.N);
    const float mean = row_sum<1024>(sum, red[0]) * inv_n;
    float sq = 0.0f;
    for (int64_t c = threadIdx.x; c < a.N; c += 1024) {
        const float d = to_f(in[c]) - mean;
        sq = fmaf(d, d, sq);
    }
    const float rstd = rsqrtf(row_sum<1024>(sq, red[1]) * inv_n + a.eps);
    if (threadIdx.x == 0) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
    }
    for (int64_t c = threadIdx.x; c < a.N; c += 1024) {
        float g[1], b[1];
        load_param<1>(a.gamma, a.p32, c, 1.0f, false, g);
        load_param<1>(a.beta, a.p32, c, 0.0f, false, b);
        static_cast<T*>(a.Y)[row * a.N + c] = from_f<T>(fmaf((to_f(in[c]) - mean) * rstd, g[0], b[0]));
    }
}

// ------------------------------------------------------------------ backward
struct BwdArgs {
    const void *dY, *S, *gamma, *dS;
    const float *mean, *rstd;
    void* dX;
    float* partial;   // [gridDim.x][2][N]: this CTA's sums of dY xh and of dY (NULL: not wanted)
    int64_t T, N;
    int p32, pvec;
};

constexpr int BWD_THREADS_PER_SM = 512;   // 128 registers a thread: 32 column sums, 16 gammas, a row's values

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src)
{
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES < 4 ? 4 : BYTES)
                     : "memory");
}

// Persistent: a block (or, TPR = 32, a warp) takes rows r, r + stride, ...
// Each thread owns the same NV x VW columns of every row and keeps their two
// sums in registers.  It copies its own columns of the rows ahead into its own
// shared-memory slots (cp.async, DEPTH rows in flight), so the pipeline needs
// no barrier; the only one per row is the row sums'.
template <typename T, int VW, int TPR, int NV>
struct BwdShape {
    static constexpr int THREADS = TPR == 32 ? 256 : TPR;
    static constexpr int CTAS = BWD_THREADS_PER_SM / THREADS;
    static constexpr int ROWS = THREADS / TPR;
    static constexpr int SLOT = sizeof(T) * VW < 4 ? 4 : sizeof(T) * VW;
    static constexpr int STAGE = THREADS * NV * SLOT * 3;       // dY, S, dS of one row (per warp / block)
    static constexpr int FIT = 192 * 1024 / CTAS / STAGE;
    static constexpr int DEPTH = FIT > 4 ? 4 : FIT;
    static constexpr int RED = ROWS > 1 ? ROWS * TPR * NV * VW * 4 : 0;   // the warps' column sums at the end
    static constexpr int RING = STAGE * DEPTH;
    static constexpr int SMEM = RING > RED ? RING : RED;
};

template <typename T, int VW, int TPR, int NV>
__global__ void __launch_bounds__(BwdShape<T, VW, TPR, NV>::THREADS, BwdShape<T, VW, TPR, NV>::CTAS)
    norm_bwd_kernel(const BwdArgs a)
{
    using Sh = BwdShape<T, VW, TPR, NV>;
    constexpr int THREADS = Sh::THREADS, ROWS = Sh::ROWS, DEPTH = Sh::DEPTH, SLOT = Sh::SLOT;
    constexpr bool ASYNC = sizeof(T) * VW >= 4;   // cp.async copies at least 4 bytes
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 red[2][TPR <= 32 ? 1 : TPR / 32];
    const int t = threadIdx.x % TPR;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * ROWS;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / TPR;
    const uint32_t slot0 = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + threadIdx.x * SLOT;
    const T* dy_p = static_cast<const T*>(a.dY);
    const T* s_p = static_cast<const T*>(a.S);
    const T* ds_p = static_cast<const T*>(a.dS);

    auto slot = [&](int stage, int tensor, int i) -> uint32_t {
        return static_cast<uint32_t>(((stage * 3 + tensor) * NV + i) * (THREADS * SLOT));
    };
    auto fetch = [&](int64_t row, int stage) {
        if (row < a.T) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = static_cast<int64_t>(i * TPR + t) * VW;
                if (c < a.N) {
                    const int64_t at = row * a.N + c;
                    if (ASYNC) {
                        copy_async<sizeof(T) * VW>(slot0 + slot(stage, 0, i), dy_p + at);
                        copy_async<sizeof(T) * VW>(slot0 + slot(stage, 1, i), s_p + at);
                        if (ds_p != nullptr)
                            copy_async<sizeof(T) * VW>(slot0 + slot(stage, 2, i), ds_p + at);
                    } else {
                        uint8_t* q = smem + threadIdx.x * SLOT;
                        const Vec<T, VW> d = load_stream<T, VW>(dy_p + at), x = load_stream<T, VW>(s_p + at);
                        *reinterpret_cast<Vec<T, VW>*>(q + slot(stage, 0, i)) = d;
                        *reinterpret_cast<Vec<T, VW>*>(q + slot(stage, 1, i)) = x;
                        if (ds_p != nullptr)
                            *reinterpret_cast<Vec<T, VW>*>(q + slot(stage, 2, i)) = load_stream<T, VW>(ds_p + at);
                    }
                }
            }
        }
        if (ASYNC)
            asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto slot_vec = [&](int stage, int tensor, int i) -> Vec<T, VW> {
        return *reinterpret_cast<const Vec<T, VW>*>(smem + threadIdx.x * SLOT + slot(stage, tensor, i));
    };

    float g[NV][VW], sum_g[NV][VW], sum_b[NV][VW];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = static_cast<int64_t>(i * TPR + t) * VW;
#pragma unroll
        for (int j = 0; j < VW; ++j)
            g[i][j] = sum_g[i][j] = sum_b[i][j] = 0.0f;
        if (c < a.N)
            load_param<VW>(a.gamma, a.p32, c, 1.0f, a.pvec, g[i]);
    }
#pragma unroll
    for (int d = 0; d < DEPTH - 1; ++d)
        fetch(first + d * stride, d);

    const float inv_n = 1.0f / static_cast<float>(a.N);
    int stage = 0, par = 0;
    float mean = 0.0f, rstd = 0.0f;
    if (first < a.T) {
        mean = __ldg(a.mean + first);
        rstd = __ldg(a.rstd + first);
    }
    for (int64_t row = first; row < a.T; row += stride) {
        const int64_t ahead = row + (DEPTH - 1) * stride;
        fetch(ahead, stage == 0 ? DEPTH - 1 : stage - 1);
        const int64_t next = row + stride;
        float mean_n = 0.0f, rstd_n = 0.0f;
        if (next < a.T) {
            mean_n = __ldg(a.mean + next);
            rstd_n = __ldg(a.rstd + next);
        }
        if (ASYNC)
            asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
        float xh[NV][VW], gy[NV][VW];
        float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = static_cast<int64_t>(i * TPR + t) * VW;
#pragma unroll
            for (int j = 0; j < VW; ++j)
                xh[i][j] = gy[i][j] = 0.0f;
            if (c < a.N) {
                const Vec<T, VW> d = slot_vec(stage, 0, i), s = slot_vec(stage, 1, i);
#pragma unroll
                for (int j = 0; j < VW; ++j) {
                    const float dy = to_f(d.e[j]);
                    xh[i][j] = (to_f(s.e[j]) - mean) * rstd;
                    sum_g[i][j] = fmaf(dy, xh[i][j], sum_g[i][j]);
                    sum_b[i][j] += dy;
                    gy[i][j] = dy * g[i][j];
                    c1 += gy[i][j];
                    c2 = fmaf(gy[i][j], xh[i][j], c2);
                }
            }
        }
        c1 = warp_sum(c1);
        c2 = warp_sum(c2);
        if (TPR > 32) {
            // two buffers: a warp may still read one while the next row's sums are written
            if ((threadIdx.x & 31) == 0)
                red[par][threadIdx.x >> 5] = make_float2(c1, c2);
            __syncthreads();
            c1 = c2 = 0.0f;
#pragma unroll
            for (int w = 0; w < TPR / 32; ++w) {
                const float2 v = red[par][w];
                c1 += v.x;
                c2 += v.y;
            }
            par ^= 1;
        }
        c1 *= inv_n;
        c2 *= inv_n;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = static_cast<int64_t>(i * TPR + t) * VW;
            if (c < a.N) {
                Vec<T, VW> o;
                float add[VW];
#pragma unroll
                for (int j = 0; j < VW; ++j)
                    add[j] = 0.0f;
                if (ds_p != nullptr) {
                    const Vec<T, VW> e = slot_vec(stage, 2, i);
#pragma unroll
                    for (int j = 0; j < VW; ++j)
                        add[j] = to_f(e.e[j]);
                }
#pragma unroll
                for (int j = 0; j < VW; ++j)
                    o.e[j] = from_f<T>(fmaf(rstd, fmaf(-xh[i][j], c2, gy[i][j] - c1), add[j]));
                store_vec<T, VW>(static_cast<T*>(a.dX) + row * a.N + c, o);
            }
        }
        mean = mean_n;
        rstd = rstd_n;
        stage = stage + 1 == DEPTH ? 0 : stage + 1;
    }
    if (ASYNC)
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (a.partial == nullptr)
        return;
    float* out = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * a.N;
    if (ROWS == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = static_cast<int64_t>(i * TPR + t) * VW;
            if (c < a.N) {
#pragma unroll
                for (int j = 0; j < VW; ++j) {
                    out[c + j] = sum_g[i][j];
                    out[a.N + c + j] = sum_b[i][j];
                }
            }
        }
        return;
    }
    // several warps per block: their sums meet in shared memory, warp order
    float* acc = reinterpret_cast<float*>(smem);
    const int span = TPR * NV * VW;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VW; ++j)
                acc[(threadIdx.x / TPR) * span + (i * TPR + t) * VW + j] = which ? sum_b[i][j] : sum_g[i][j];
        __syncthreads();
        for (int64_t c = threadIdx.x; c < a.N; c += THREADS) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < ROWS; ++w)
                v += acc[w * span + c];
            out[which * a.N + c] = v;
        }
    }
}

// dgamma, dbeta from the CTAs' sums: 32 columns per block, 16 strands of CTAs
// per column, joined in order.
__global__ void __launch_bounds__(512) norm_sums_kernel(const float* partial, int ctas, int64_t N, float* dgamma,
                                                        float* dbeta)
{
    __shared__ float red[16][33];
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float v = 0.0f;
    if (c < N)
        for (int k = y; k < ctas; k += 16)
            v += partial[(static_cast<int64_t>(k) * 2 + blockIdx.y) * N + c];
    red[y][lane] = v;
    __syncthreads();
    if (y == 0 && c < N) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            s += red[i][lane];
        (blockIdx.y ? dbeta : dgamma)[c] = s;
    }
}

// Rows too long for a block's registers: dX by one block per row (two passes),
// the column sums by a second sweep.
template <typename T>
__global__ void __launch_bounds__(1024) norm_bwd_long_kernel(const BwdArgs a)
{
    __shared__ float red[2][32];
    const int64_t row = blockIdx.x;
    const T* dy = static_cast<const T*>(a.dY) + row * a.N;
    const T* s = static_cast<const T*>(a.S) + row * a.N;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float c1 = 0.0f, c2 = 0.0f;
    for (int64_t c = threadIdx.x; c < a.N; c += 1024) {
        float g[1];
        load_param<1>(a.gamma, a.p32, c, 1.0f, false, g);
        const float gy = to_f(dy[c]) * g[0];
        c1 += gy;
        c2 = fmaf(gy, (to_f(s[c]) - mean) * rstd, c2);
    }
    const float inv_n = 1.0f / static_cast<float>(a.N);
    c1 = row_sum<1024>(c1, red[0]) * inv_n;
    c2 = row_sum<1024>(c2, red[1]) * inv_n;
    for (int64_t c = threadIdx.x; c < a.N; c += 1024) {
        float g[1];
        load_param<1>(a.gamma, a.p32, c, 1.0f, false, g);
        const float add = a.dS == nullptr ? 0.0f : to_f(static_cast<const T*>(a.dS)[row * a.N + c]);
        const float xh = (to_f(s[c]) - mean) * rstd;
        static_cast<T*>(a.dX)[row * a.N + c] =
            from_f<T>(fmaf(rstd, fmaf(-xh, c2, to_f(dy[c]) * g[0] - c1), add));
    }
}

template <typename T>
__global__ void __launch_bounds__(128) norm_columns_kernel(const BwdArgs a, int chunks)
{
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
    if (c >= a.N)
        return;
    const int64_t r0 = a.T * blockIdx.y / chunks, r1 = a.T * (blockIdx.y + 1) / chunks;
    float sg = 0.0f, sb = 0.0f;
    for (int64_t r = r0; r < r1; ++r) {
        const float dy = to_f(static_cast<const T*>(a.dY)[r * a.N + c]);
        const float xh = (to_f(static_cast<const T*>(a.S)[r * a.N + c]) - __ldg(a.mean + r)) * __ldg(a.rstd + r);
        sg = fmaf(dy, xh, sg);
        sb += dy;
    }
    float* out = a.partial + static_cast<int64_t>(blockIdx.y) * 2 * a.N;
    out[c] = sg;
    out[a.N + c] = sb;
}

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <typename T, int VW, int TPR, int NV>
int fwd(const FwdArgs& a, cudaStream_t s)
{
    constexpr int threads = TPR < 128 ? 128 : TPR;
    constexpr int rows = threads / TPR;
    norm_fwd_kernel<T, VW, TPR, NV><<<static_cast<unsigned>((a.T + rows - 1) / rows), threads, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

// Threads and vectors per row by the row's vectors: a warp up to 128 vectors
// (no block barrier), then blocks of four vectors a thread.
template <typename T, int VW>
int fwd_any(const FwdArgs& a, cudaStream_t s)
{
    const int64_t v = (a.N + VW - 1) / VW;
    if (v <= 32)
        return fwd<T, VW, 32, 1>(a, s);
    if (v <= 64)
        return fwd<T, VW, 32, 2>(a, s);
    if (v <= 128)
        return fwd<T, VW, 32, 4>(a, s);
    if (v <= 256)
        return fwd<T, VW, 128, 2>(a, s);
    if (v <= 512)
        return fwd<T, VW, 128, 4>(a, s);
    if (v <= 1024)
        return fwd<T, VW, 256, 4>(a, s);
    if (v <= 2048)
        return fwd<T, VW, 512, 4>(a, s);
    if (v <= 4096)
        return fwd<T, VW, 1024, 4>(a, s);
    if (VW <= 2 && v <= 8192)
        return fwd<T, VW <= 2 ? VW : 1, 1024, 8>(a, s);
    norm_fwd_long_kernel<T><<<static_cast<unsigned>(a.T), 1024, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

// Columns a block of 512 threads holds 16 of in each thread's registers.
constexpr int64_t BWD_MAX_N = 8192;

// (threads per row, rows per CTA, CTAs per SM) of a width: one rule for every
// type, so that the workspace can be sized without knowing it.
void bwd_shape(int64_t N, int& tpr, int& ctas_per_sm)
{
    tpr = N <= 512 ? 32 : N <= 2048 ? 128 : N <= 4096 ? 256 : 512;
    ctas_per_sm = BWD_THREADS_PER_SM / (tpr == 32 ? 256 : tpr);
}

template <typename T, int VW, int TPR, int NV>
int bwd(const BwdArgs& a, int ctas, cudaStream_t s)
{
    using Sh = BwdShape<T, VW, TPR, NV>;
    static_assert(TPR * NV * VW <= BWD_MAX_N && Sh::DEPTH >= 2, "a row fits, two rows in flight");
    if (cudaFuncSetAttribute(norm_bwd_kernel<T, VW, TPR, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Sh::SMEM) != cudaSuccess)
        return -1;
    norm_bwd_kernel<T, VW, TPR, NV><<<ctas, Sh::THREADS, Sh::SMEM, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

template <typename T, int VW>
int bwd_any(const BwdArgs& a, int ctas, cudaStream_t s)
{
    constexpr int F = 16 / VW;   // vectors of 16 columns
    if (a.N <= 256)
        return bwd<T, VW, 32, F / 2>(a, ctas, s);
    if (a.N <= 512)
        return bwd<T, VW, 32, F>(a, ctas, s);
    if (a.N <= 1024)
        return bwd<T, VW, 128, F / 2>(a, ctas, s);
    if (a.N <= 2048)
        return bwd<T, VW, 128, F>(a, ctas, s);
    if (a.N <= 4096)
        return bwd<T, VW, 256, F>(a, ctas, s);
    return bwd<T, VW, 512, F>(a, ctas, s);
}

}  // namespace norm

int launch_norm_fwd(const NormFwd& n, int sms, cudaStream_t s)
{
    using namespace norm;
    (void)sms;
    FwdArgs a{n.X, n.R, n.gamma, n.beta, n.Y, n.S, n.mean, n.rstd, n.T, n.N, n.eps, n.p32 ? 1 : 0, 0};
    a.pvec = aligned_to(n.gamma, 16) && aligned_to(n.beta, 16) ? 1 : 0;
    const size_t e = n.f32 ? 4 : 2;
    auto fits = [&](size_t bytes) {   // every row of every tensor starts on a multiple of `bytes`
        return (n.N * e) % bytes == 0 && aligned_to(n.X, bytes) && aligned_to(n.R, bytes) && aligned_to(n.Y, bytes) &&
               aligned_to(n.S, bytes);
    };
    if (n.f32)
        return fits(16) ? fwd_any<float, 4>(a, s) : fwd_any<float, 1>(a, s);
    if (fits(16))
        return fwd_any<__nv_bfloat16, 8>(a, s);
    return fits(4) ? fwd_any<__nv_bfloat16, 2>(a, s) : fwd_any<__nv_bfloat16, 1>(a, s);
}

int norm_bwd_ctas(int64_t T, int64_t N, int sms)
{
    using namespace norm;
    if (N > BWD_MAX_N)   // row chunks of the column sweep
        return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(64, (T + 31) / 32)));
    int tpr = 0, per_sm = 0;
    bwd_shape(N, tpr, per_sm);
    const int rows = tpr == 32 ? 8 : 1;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((T + rows - 1) / rows, int64_t(sms) * per_sm)));
}

int launch_norm_bwd(const NormBwd& n, int sms, cudaStream_t s)
{
    using namespace norm;
    const int ctas = norm_bwd_ctas(n.T, n.N, sms);
    BwdArgs a{n.dY, n.S, n.gamma, n.dS, n.mean, n.rstd, n.dX, n.dgamma ? n.partial : nullptr, n.T, n.N,
              n.p32 ? 1 : 0, aligned_to(n.gamma, 16) ? 1 : 0};
    int launches = 1;
    if (n.N > BWD_MAX_N) {
        if (n.f32)
            norm_bwd_long_kernel<float><<<static_cast<unsigned>(n.T), 1024, 0, s>>>(a);
        else
            norm_bwd_long_kernel<__nv_bfloat16><<<static_cast<unsigned>(n.T), 1024, 0, s>>>(a);
        if (n.dgamma) {
            const dim3 grid(static_cast<unsigned>((n.N + 127) / 128), static_cast<unsigned>(ctas));
            if (n.f32)
                norm_columns_kernel<float><<<grid, 128, 0, s>>>(a, ctas);
            else
                norm_columns_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>(a, ctas);
            ++launches;
        }
    } else {
        const size_t e = n.f32 ? 4 : 2;
        auto fits = [&](size_t bytes) {
            return (n.N * e) % bytes == 0 && aligned_to(n.dY, bytes) && aligned_to(n.S, bytes) &&
                   aligned_to(n.dS, bytes) && aligned_to(n.dX, bytes);
        };
        int rc;
        if (n.f32)
            rc = fits(16) ? bwd_any<float, 4>(a, ctas, s) : bwd_any<float, 1>(a, ctas, s);
        else if (fits(16))
            rc = bwd_any<__nv_bfloat16, 8>(a, ctas, s);
        else
            rc = fits(4) ? bwd_any<__nv_bfloat16, 2>(a, ctas, s) : bwd_any<__nv_bfloat16, 1>(a, ctas, s);
        if (rc != 0)
            return -1;
    }
    if (n.dgamma) {
        const dim3 grid(static_cast<unsigned>((n.N + 31) / 32), 2);
        norm_sums_kernel<<<grid, 512, 0, s>>>(n.partial, ctas, n.N, n.dgamma, n.dbeta);
        ++launches;
    }
    return cudaGetLastError() == cudaSuccess ? launches : -1;
}

}  // namespace tffn
