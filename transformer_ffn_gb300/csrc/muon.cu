// muon.cu -- muon_orthogonalize beside its large products: the Frobenius norm,
// the scaled fp16 copy that the Newton-Schulz products start from, the dense
// copy of a result whose rows the products stored padded, and the whole
// iteration for matrices with a small side.
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

// One entry's factor from its blocks' sums: X = (G before) factor = scale G /
// (norm + eps).  A norm past 2^60 is first brought down, so that neither number
// leaves fp32's normal range.  Called by a whole block.
__device__ __forceinline__ float2 entry_factor(const double* part, int blocks, float scale, float eps)
{
    __shared__ double red[THREADS / 32];
    __shared__ float2 result;
    double d = 0.0;
    for (int k = threadIdx.x; k < blocks; k += THREADS)
        d += part[k];
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
        const double norm = sqrt(d) + static_cast<double>(eps);
        const double pre = norm > 0x1p60 ? 0x1p-60 : 1.0;
        result = make_float2(static_cast<float>(pre),
                             static_cast<float>(static_cast<double>(scale) / (norm * pre)));
    }
    __syncthreads();
    return result;
}

// X[r][c] = fp16(scale G[r][c] / (norm + eps)), zero in the padding columns.
template <typename T>
__global__ void __launch_bounds__(THREADS) muon_pack_kernel(const T* G, int64_t m, int64_t n, const double* part,
                                                            int blocks, float scale, float eps, __half* X, int64_t ld,
                                                            int vec)
{
    const T* g = G + blockIdx.y * m * n;
    __half* x = X + blockIdx.y * m * ld;
    const float2 fs = entry_factor(part + static_cast<int64_t>(blockIdx.y) * blocks, blocks, scale, eps);
    const float f0 = fs.x, f = fs.y;
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

// ---- small sides.  With at most 64 rows (or columns) the iteration runs on the
// side x side matrix A = X X^T alone, in fp32: X_k = Q_k X_0 with Q_{k+1} = P_k
// Q_k, P_k = a I + b A_k + c A_k^2 and A_{k+1} = P_k A_k P_k (polynomials of A_0
// commute, so all of these are symmetric).  Two kernels beside the norm: A_0 in
// parts of the long side, and Q with its product.  Every block of the second
// runs the whole iteration (18 products of side^3, each about 3 us at 64 and
// bound by shared-memory loads and their latency) before its share of the
// product, which costs nothing beside handing Q over.  Measured against the
// tensor-core products' fifteen dependent phases: 16 x 300 22 us (63), 32 x 2000
// 25 (80), 64 x 64 55 (60), 64 x 4096 72 (95), three of 5288 x 48 86 (111); the
// time grows with the side's cube, so 64 is where it ends.  And fp32 keeps what
// fp16 loses where few entries make a matrix (3e-3 of its norm with 16 rows).
constexpr int CHUNK = 64;   // long-side elements in shared memory at a time

// One chunk of an entry, [S short][CHUNK long], scaled; zero outside.
template <typename T, int S>
__device__ __forceinline__ void load_chunk(const T* g, bool tall, int side, int64_t len, int64_t c0, float2 fs,
                                           float (*x)[CHUNK + 4])
{
    for (int i = threadIdx.x; i < S * CHUNK; i += THREADS) {
        // neighbouring threads read neighbouring elements either way
        const int k = tall ? i % S : i / CHUNK, c = tall ? i / S : i % CHUNK;
        float v = 0.0f;
        if (k < side && c0 + c < len)
            v = to_f(g[tall ? (c0 + c) * side + k : k * len + c0 + c]);
        x[k][c] = v * fs.x * fs.y;
    }
}

// A thread's MT x MT block of the S x S result, rows i0.., columns j0..
template <int S>
struct Tile {
    static constexpr int MT = S / 16;   // 16 x 16 threads
    int i0, j0;
    __device__ __forceinline__ Tile() : i0((threadIdx.x / 16) * MT), j0((threadIdx.x % 16) * MT) {}
};

// part[entry][chunk set][S][S]: partial sums of X X^T.
template <typename T, int S>
__global__ void __launch_bounds__(THREADS) muon_small_gram_kernel(const T* G, bool tall, int side, int64_t len,
                                                                  const double* norm, int blocks, float eps,
                                                                  float* part)
{
    __shared__ float x[S][CHUNK + 4];
    constexpr int MT = Tile<S>::MT;
    const Tile<S> t;
    const T* g = G + blockIdx.y * (static_cast<int64_t>(side) * len);
    const float2 fs = entry_factor(norm + static_cast<int64_t>(blockIdx.y) * blocks, blocks, 1.0f, eps);
    float acc[MT][MT] = {};
    for (int64_t c0 = static_cast<int64_t>(blockIdx.x) * CHUNK; c0 < len;
         c0 += static_cast<int64_t>(gridDim.x) * CHUNK) {
        __syncthreads();
        load_chunk<T, S>(g, tall, side, len, c0, fs, x);
        __syncthreads();
        for (int c = 0; c < CHUNK; c += 4) {
            float4 a[MT], b[MT];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                a[i] = *reinterpret_cast<const float4*>(&x[t.i0 + i][c]);
                b[i] = *reinterpret_cast<const float4*>(&x[t.j0 + i][c]);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < MT; ++j)
                    acc[i][j] += a[i].x * b[j].x + a[i].y * b[j].y + a[i].z * b[j].z + a[i].w * b[j].w;
        }
    }
    float* out = part + (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * S * S;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
            out[(t.i0 + i) * S + t.j0 + j] = acc[i][j];
}

template <int S>
using Square = float[S][S + 4];   // rows stay on 16-byte boundaries

// MT consecutive values of a row, from a multiple of MT.
template <int MT>
__device__ __forceinline__ void load_run(const float* p, float (&v)[MT])
{
    static_assert(MT == 2 || MT == 4, "one shared-memory load");
    if constexpr (MT == 4) {
        const float4 x = *reinterpret_cast<const float4*>(p);
        v[0] = x.x;
        v[1] = x.y;
        v[2] = x.z;
        v[3] = x.w;
    } else {
        const float2 x = *reinterpret_cast<const float2*>(p);
        v[0] = x.x;
        v[1] = x.y;
    }
}

// out = alpha A B + beta C + diag I of symmetric matrices (C nullable).
template <int S>
__device__ __forceinline__ void product(const Square<S>& A, const Square<S>& B, Square<S>& out, float alpha,
                                        float beta, const Square<S>* C, float diag)
{
    constexpr int MT = Tile<S>::MT;
    const Tile<S> t;
    float acc[MT][MT] = {};
#pragma unroll 8
    for (int k = 0; k < S; ++k) {
        float a[MT], b[MT];
        load_run(&A[k][t.i0], a);   // row k for column k: A is symmetric
        load_run(&B[k][t.j0], b);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j)
                acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const int r = t.i0 + i, c = t.j0 + j;
            float v = alpha * acc[i][j] + (r == c ? diag : 0.0f);
            if (C != nullptr)
                v = fmaf(beta, (*C)[r][c], v);
            out[r][c] = v;
        }
    __syncthreads();
}

template <int S>
struct SmallShared {
    Square<S> a, p, t, q[2];
    float x[S][CHUNK + 4];
};

template <typename T, int S>
__global__ void __launch_bounds__(THREADS) muon_small_apply_kernel(const T* G, bool tall, int side, int64_t len,
                                                                   const double* norm, int blocks, float eps,
                                                                   const float* part, int parts, int steps, float ca,
                                                                   float cb, float cc, __nv_bfloat16* out)
{
    extern __shared__ __align__(16) uint8_t smem[];
    SmallShared<S>& sh = *reinterpret_cast<SmallShared<S>*>(smem);
    constexpr int MT = Tile<S>::MT;
    const Tile<S> t;
    const int64_t entry = static_cast<int64_t>(blockIdx.y) * side * len;
    const float2 fs = entry_factor(norm + static_cast<int64_t>(blockIdx.y) * blocks, blocks, 1.0f, eps);
    const float* src = part + static_cast<int64_t>(blockIdx.y) * parts * S * S;
    for (int i = threadIdx.x; i < S * S; i += THREADS) {
        float v = 0.0f;
        for (int k = 0; k < parts; ++k)
            v += __ldg(src + static_cast<int64_t>(k) * S * S + i);
        sh.a[i / S][i % S] = v;
        sh.q[0][i / S][i % S] = i / S == i % S ? 1.0f : 0.0f;
    }
    __syncthreads();
    int cur = 0;
    for (int k = 0; k < steps; ++k) {
        product<S>(sh.a, sh.a, sh.p, cc, cb, &sh.a, ca);
        product<S>(sh.p, sh.q[cur], sh.q[cur ^ 1], 1.0f, 0.0f, nullptr, 0.0f);
        cur ^= 1;
        if (k + 1 < steps) {
            product<S>(sh.a, sh.p, sh.t, 1.0f, 0.0f, nullptr, 0.0f);
            product<S>(sh.t, sh.p, sh.a, 1.0f, 0.0f, nullptr, 0.0f);
        }
    }
    const Square<S>& Q = sh.q[cur];
    constexpr int CT = CHUNK / 16;   // long-side elements of a thread
    const int c_first = (threadIdx.x % 16) * CT;
    for (int64_t c0 = static_cast<int64_t>(blockIdx.x) * CHUNK; c0 < len;
         c0 += static_cast<int64_t>(gridDim.x) * CHUNK) {
        __syncthreads();
        load_chunk<T, S>(G + entry, tall, side, len, c0, fs, sh.x);
        __syncthreads();
        float acc[MT][CT] = {};
#pragma unroll 4
        for (int k = 0; k < S; ++k) {
            const float4 x = *reinterpret_cast<const float4*>(&sh.x[k][c_first]);
            float q[MT];
            load_run(&Q[k][t.i0], q);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                acc[i][0] = fmaf(q[i], x.x, acc[i][0]);
                acc[i][1] = fmaf(q[i], x.y, acc[i][1]);
                acc[i][2] = fmaf(q[i], x.z, acc[i][2]);
                acc[i][3] = fmaf(q[i], x.w, acc[i][3]);
            }
        }
        // through shared memory, so that neighbouring threads store neighbours
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MT; ++i)
            *reinterpret_cast<float4*>(&sh.x[t.i0 + i][c_first]) =
                make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        __syncthreads();
        for (int i = threadIdx.x; i < S * CHUNK; i += THREADS) {
            const int k = tall ? i % S : i / CHUNK, c = tall ? i / S : i % CHUNK;
            if (k < side && c0 + c < len)
                out[entry + (tall ? (c0 + c) * side + k : k * len + c0 + c)] = __float2bfloat16_rn(sh.x[k][c]);
        }
    }
}

template <typename T, int S>
int small(const T* G, int64_t batch, bool tall, int side, int64_t len, const double* norm, int blocks, float eps,
          float* part, int parts, int steps, const float* abc, __nv_bfloat16* out, int sms, cudaStream_t s)
{
    static bool ready = false;
    if (!ready && cudaFuncSetAttribute(muon_small_apply_kernel<T, S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       sizeof(SmallShared<S>)) != cudaSuccess)
        return -1;
    ready = true;
    const int64_t chunks = (len + CHUNK - 1) / CHUNK;
    const unsigned y = static_cast<unsigned>(batch);
    muon_small_gram_kernel<T, S>
        <<<dim3(static_cast<unsigned>(parts), y), THREADS, 0, s>>>(G, tall, side, len, norm, blocks, eps, part);
    // one block an SM: each runs the whole iteration
    const int64_t x = std::max<int64_t>(1, std::min<int64_t>(chunks, int64_t(sms) / batch));
    muon_small_apply_kernel<T, S><<<dim3(static_cast<unsigned>(x), y), THREADS, sizeof(SmallShared<S>), s>>>(
        G, tall, side, len, norm, blocks, eps, part, parts, steps, abc[0], abc[1], abc[2], out);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
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

int muon_norm_blocks(int64_t batch, int64_t elems, int sms)
{
    // of each entry: eight values a thread at least, at most four blocks an SM
    // for all entries together (with four for each, eight entries of 4096 x 1024
    // fp32 took 60 us instead of 29)
    return static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>(int64_t(sms) * 4 / batch, elems / (muon::THREADS * 8))));
}

int muon_small_side() { return 64; }

// Parts of the long side: enough to occupy the GPU, at most 32 (every block of
// the second kernel adds them all).
int muon_small_parts(int64_t batch, int64_t len, int sms)
{
    const int64_t chunks = (len + muon::CHUNK - 1) / muon::CHUNK;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(chunks, 32), 2 * int64_t(sms) / batch)));
}

size_t muon_small_bytes(int64_t batch, int64_t side, int64_t len, int sms)
{
    const int64_t S = side <= 32 ? 32 : 64;
    return static_cast<size_t>(batch * muon_small_parts(batch, len, sms) * S * S * 4);
}

int launch_muon_small(const void* G, bool f32, int64_t batch, int64_t m, int64_t n, const double* norm, int blocks,
                      float eps, float* part, int steps, const float* abc, void* out, int sms, cudaStream_t s)
{
    const bool tall = m > n;
    const int side = static_cast<int>(std::min(m, n));
    const int64_t len = std::max(m, n);
    const int parts = muon_small_parts(batch, len, sms);
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out);
    const float* gf = static_cast<const float*>(G);
    const __nv_bfloat16* gb = static_cast<const __nv_bfloat16*>(G);
    if (side <= 32)
        return f32 ? muon::small<float, 32>(gf, batch, tall, side, len, norm, blocks, eps, part, parts, steps, abc, o,
                                            sms, s)
                   : muon::small<__nv_bfloat16, 32>(gb, batch, tall, side, len, norm, blocks, eps, part, parts, steps,
                                                    abc, o, sms, s);
    return f32 ? muon::small<float, 64>(gf, batch, tall, side, len, norm, blocks, eps, part, parts, steps, abc, o, sms,
                                        s)
               : muon::small<__nv_bfloat16, 64>(gb, batch, tall, side, len, norm, blocks, eps, part, parts, steps, abc,
                                                o, sms, s);
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
