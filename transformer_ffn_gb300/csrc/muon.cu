// muon.cu -- the memory-bound ends of muon_orthogonalize: the Frobenius norm,
// the scaled fp16 copy that the Newton-Schulz products start from, and the
// dense copy of a result whose rows the products stored padded.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "train.h"

namespace tffn {
namespace muon {

constexpr int THREADS = 256;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
struct alignas(16) Vec {
    static constexpr int W = 16 / sizeof(T);
    T e[W];
};

// A thread's sum of squares in fp32: values past 2^40, whose squares could leave
// fp32's range, are added 2^-80 times themselves (squares below fp32's range do
// not matter beside the 1e-7 that the norm is added to).
struct Squares {
    float small = 0.0f, large = 0.0f;
    __device__ __forceinline__ void add(float x)
    {
        const bool big = fabsf(x) > 0x1p40f;
        const float y = big ? x * 0x1p-80f : x;
        const float q = y * y;
        small += big ? 0.0f : q;
        large += big ? q : 0.0f;
    }
    __device__ __forceinline__ double sum() const
    {
        return static_cast<double>(small) + static_cast<double>(large) * 0x1p160;
    }
};

// Sums of squares of one entry's `elems` values: part[entry][block].  A thread
// adds in fp32 over its own few thousand values, threads are joined in fp64.
template <typename T>
__global__ void __launch_bounds__(THREADS) muon_norm_kernel(const T* G, int64_t elems, double* part)
{
    __shared__ double red[THREADS / 32];
    const T* g = G + blockIdx.y * elems;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * THREADS;
    constexpr int W = Vec<T>::W;
    // values before the first 16-byte boundary, whole vectors, and the rest
    const int64_t mis = static_cast<int64_t>((reinterpret_cast<uintptr_t>(g) & 15u) / sizeof(T));
    const int64_t head = mis == 0 ? 0 : (W - mis < elems ? W - mis : elems);
    const int64_t vecs = (elems - head) / W;
    const Vec<T>* v = reinterpret_cast<const Vec<T>*>(g + head);
    Squares s[4];
    int64_t i = id;
    for (; i + 3 * step < vecs; i += 4 * step) {
        Vec<T> x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            x[k] = v[i + k * step];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < W; ++j)
                s[k].add(to_f(x[k].e[j]));
    }
    for (; i < vecs; i += step) {
        const Vec<T> x = v[i];
#pragma unroll
        for (int j = 0; j < W; ++j)
            s[0].add(to_f(x.e[j]));
    }
    const int64_t tail = head + vecs * W;
    for (int64_t k = id; k < head + (elems - tail); k += step) {
        s[1].add(to_f(k < head ? g[k] : g[tail + k - head]));
    }
    double d = s[0].sum() + s[1].sum() + s[2].sum() + s[3].sum();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        d += __shfl_xor_sync(0xffffffffu, d, o);
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = d;
    __syncthreads();
    if (threadIdx.x == 0) {
        d = 0.0;
        for (int k = 0; k < THREADS / 32; ++k)
            d += red[k];
        part[static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x] = d;
    }
}

// X[r][c] = fp16(scale G[r][c] / (norm + eps)), zero in the padding columns.
template <typename T>
__global__ void __launch_bounds__(THREADS) muon_pack_kernel(const T* G, int64_t m, int64_t n, const double* part,
                                                            int blocks, float scale, float eps, __half* X, int64_t ld,
                                                            int vec)
{
    __shared__ double red[THREADS / 32];
    __shared__ float factor, before;
    const T* g = G + blockIdx.y * m * n;
    __half* x = X + blockIdx.y * m * ld;
    double d = 0.0;
    for (int k = threadIdx.x; k < blocks; k += THREADS)
        d += part[static_cast<int64_t>(blockIdx.y) * blocks + k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        d += __shfl_xor_sync(0xffffffffu, d, o);
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = d;
    __syncthreads();
    if (threadIdx.x == 0) {
        d = 0.0;
        for (int k = 0; k < THREADS / 32; ++k)
            d += red[k];
        // X = (G before) factor: a norm past 2^60 is first brought down, so that
        // neither number leaves fp32's normal range
        const double norm = sqrt(d) + static_cast<double>(eps);
        const double pre = norm > 0x1p60 ? 0x1p-60 : 1.0;
        before = static_cast<float>(pre);
        factor = static_cast<float>(static_cast<double>(scale) / (norm * pre));
    }
    __syncthreads();
    const float f = factor, f0 = before;
    const int64_t per_row = ld / 8;
    const int64_t total = m * per_row;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * THREADS) {
        const int64_t r = i / per_row, c = (i - r * per_row) * 8;
        const T* src = g + r * n + c;
        float v[8];
        if (vec != 0 && c + 8 <= n) {
            constexpr int W = Vec<T>::W;
#pragma unroll
            for (int k = 0; k < 8 / W; ++k) {
                const Vec<T> q = reinterpret_cast<const Vec<T>*>(src)[k];
#pragma unroll
                for (int j = 0; j < W; ++j)
                    v[k * W + j] = to_f(q.e[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = c + j < n ? to_f(src[j]) : 0.0f;
        }
        __half2 o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[j] = __floats2half2_rn(v[2 * j] * f0 * f, v[2 * j + 1] * f0 * f);
        *reinterpret_cast<uint4*>(x + r * ld + c) = *reinterpret_cast<const uint4*>(o);
    }
}

// 16-bit rows of stride ld to dense rows of n.
__global__ void __launch_bounds__(THREADS) muon_unpack_kernel(const uint16_t* X, int64_t rows, int64_t n, int64_t ld,
                                                              uint16_t* out)
{
    const int64_t total = rows * n;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * THREADS) {
        const int64_t r = i / n;
        out[i] = X[r * ld + (i - r * n)];
    }
}

template <typename T>
int pack(const void* G, int64_t batch, int64_t m, int64_t n, const double* part, int blocks, float scale, float eps,
         void* X, int64_t ld, int sms, cudaStream_t s)
{
    const bool vec = (n * sizeof(T)) % 16 == 0 && (reinterpret_cast<uintptr_t>(G) & 15u) == 0;
    const int64_t need = (m * (ld / 8) + THREADS - 1) / THREADS;
    const int64_t most = std::max<int64_t>(1, int64_t(sms) * 8 / batch);
    const dim3 grid(static_cast<unsigned>(std::min(need, most)), static_cast<unsigned>(batch));
    muon_pack_kernel<T><<<grid, THREADS, 0, s>>>(static_cast<const T*>(G), m, n, part, blocks, scale, eps,
                                                 static_cast<__half*>(X), ld, vec ? 1 : 0);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace muon

int muon_norm_blocks(int64_t elems, int sms)
{
    // eight values a thread at least, at most four blocks an SM
    return static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>(int64_t(sms) * 4, elems / (muon::THREADS * 8))));
}

int launch_muon_norm(const void* G, bool f32, int64_t batch, int64_t elems, double* part, int blocks, cudaStream_t s)
{
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(batch));
    if (f32)
        muon::muon_norm_kernel<float><<<grid, muon::THREADS, 0, s>>>(static_cast<const float*>(G), elems, part);
    else
        muon::muon_norm_kernel<__nv_bfloat16>
            <<<grid, muon::THREADS, 0, s>>>(static_cast<const __nv_bfloat16*>(G), elems, part);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

int launch_muon_pack(const void* G, bool f32, int64_t batch, int64_t m, int64_t n, const double* part, int blocks,
                     float scale, float eps, void* X, int64_t ld, int sms, cudaStream_t s)
{
    return f32 ? muon::pack<float>(G, batch, m, n, part, blocks, scale, eps, X, ld, sms, s)
               : muon::pack<__nv_bfloat16>(G, batch, m, n, part, blocks, scale, eps, X, ld, sms, s);
}

int launch_muon_unpack(const void* X, int64_t batch, int64_t m, int64_t n, int64_t ld, void* out, int sms,
                       cudaStream_t s)
{
    const int64_t need = (batch * m * n + muon::THREADS - 1) / muon::THREADS;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(need, int64_t(sms) * 8));
    muon::muon_unpack_kernel<<<grid, muon::THREADS, 0, s>>>(static_cast<const uint16_t*>(X), batch * m, n, ld,
                                                            static_cast<uint16_t*>(out));
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace tffn
