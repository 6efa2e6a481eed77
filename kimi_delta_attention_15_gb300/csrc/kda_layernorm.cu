// Layer norm over rows, forward and backward, statistics and sums in fp32.
//   y  = (x - mean) rstd w + b
//   dx = rstd (a - mean(a) - xh mean(a xh)),  a = dy w,  xh = (x - mean) rstd
//   dw = sum_rows dy xh,  db = sum_rows dy
#include <cmath>
#include <cstdio>
#include "kda_internal.cuh"

namespace kda {
void set_last_error_text(const char* msg);

namespace {
constexpr int kThreads = 256;
constexpr int kPartRows = 304;   // most row blocks of the partial sums of dw, db

template <typename T> __device__ __forceinline__ float ld(const T* p, size_t i);
template <> __device__ __forceinline__ float ld<uint16_t>(const uint16_t* p, size_t i) { return bf2f(p[i]); }
template <> __device__ __forceinline__ float ld<float>(const float* p, size_t i) { return p[i]; }
__device__ __forceinline__ void st(uint16_t* p, size_t i, float x) { p[i] = f2bf(x); }
__device__ __forceinline__ void st(float* p, size_t i, float x) { p[i] = x; }

// sum over the block, the same value in every thread
__device__ __forceinline__ float block_sum(float x, float* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < (int)blockDim.x / 32; ++i) s += buf[i];
    return s;
}

// One row for each block, read three times (from the cache after the first).
template <typename T>
__global__ void __launch_bounds__(kThreads)
    layernorm_fwd_kernel(const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ b,
                         T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd, int64_t rows, int width,
                         float eps) {
    __shared__ float buf[32];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T* xr = x + r * width;
        float s = 0.0f;
        for (int c = threadIdx.x; c < width; c += kThreads) s += ld(xr, c);
        const float mu = block_sum(s, buf) / (float)width;
        s = 0.0f;
        for (int c = threadIdx.x; c < width; c += kThreads) {
            const float d = ld(xr, c) - mu;
            s += d * d;
        }
        const float rs = rsqrtf(block_sum(s, buf) / (float)width + eps);
        for (int c = threadIdx.x; c < width; c += kThreads)
            st(y + r * width, c, (ld(xr, c) - mu) * rs * (w ? w[c] : 1.0f) + (b ? b[c] : 0.0f));
        if (threadIdx.x == 0) {
            if (mean) mean[r] = mu;
            if (rstd) rstd[r] = rs;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    layernorm_dx_kernel(const T* __restrict__ x, const T* __restrict__ dy, const float* __restrict__ w,
                        const float* __restrict__ mean, const float* __restrict__ rstd, T* __restrict__ dx, int64_t rows,
                        int width) {
    __shared__ float buf[32];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const float mu = mean[r], rs = rstd[r];
        float s1 = 0.0f, s2 = 0.0f;
        for (int c = threadIdx.x; c < width; c += kThreads) {
            const float a = ld(dy, r * width + c) * (w ? w[c] : 1.0f);
            s1 += a;
            s2 += a * ((ld(x, r * width + c) - mu) * rs);
        }
        s1 = block_sum(s1, buf) / (float)width;
        s2 = block_sum(s2, buf) / (float)width;
        for (int c = threadIdx.x; c < width; c += kThreads) {
            const float a = ld(dy, r * width + c) * (w ? w[c] : 1.0f);
            st(dx + r * width, c, rs * (a - s1 - (ld(x, r * width + c) - mu) * rs * s2));
        }
    }
}

// Partial sums of dw and db: block (i, j) takes 256 columns and every gridDim.y-th row.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    layernorm_dw_kernel(const T* __restrict__ x, const T* __restrict__ dy, const float* __restrict__ mean,
                        const float* __restrict__ rstd, float* __restrict__ part, int64_t rows, int width) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= width) return;
    float dw = 0.0f, db = 0.0f;
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
        const float g = ld(dy, r * width + c);
        dw += g * ((ld(x, r * width + c) - mean[r]) * rstd[r]);
        db += g;
    }
    part[((size_t)blockIdx.y * 2) * width + c] = dw;
    part[((size_t)blockIdx.y * 2 + 1) * width + c] = db;
}

__global__ void __launch_bounds__(kThreads)
    layernorm_reduce_kernel(const float* __restrict__ part, int n, int width, float* __restrict__ dw, float* __restrict__ db) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= width) return;
    float a = 0.0f, b = 0.0f;
    for (int i = 0; i < n; ++i) {
        a += part[((size_t)i * 2) * width + c];
        b += part[((size_t)i * 2 + 1) * width + c];
    }
    if (dw) dw[c] = a;
    if (db) db[c] = b;
}

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

kda_status launched(const char* where) {
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return KDA_OK;
    char msg[160];
    snprintf(msg, sizeof(msg), "%s: %s (%d)", where, cudaGetErrorString(e), (int)e);
    set_last_error_text(msg);
    return KDA_ERR_CUDA;
}

bool valid_size(long long rows, long long width) {
    return rows >= 0 && width >= 1 && width <= (1LL << 20) && rows <= (1LL << 40) / width;
}

unsigned part_rows(long long rows) { return (unsigned)(rows < kPartRows ? rows : kPartRows); }

template <typename T>
void fwd(long long rows, int width, float eps, const void* x, const float* w, const float* b, void* y, float* mean,
         float* rstd, cudaStream_t s) {
    const unsigned grid = (unsigned)(rows < (1LL << 30) ? rows : (1LL << 30));
    layernorm_fwd_kernel<T><<<grid, kThreads, 0, s>>>(static_cast<const T*>(x), w, b, static_cast<T*>(y), mean, rstd, rows,
                                                      width, eps);
}

template <typename T>
void bwd(long long rows, int width, const void* x, const void* dy, const float* w, const float* mean, const float* rstd,
         void* dx, float* part, cudaStream_t s) {
    const unsigned grid = (unsigned)(rows < (1LL << 30) ? rows : (1LL << 30));
    layernorm_dx_kernel<T><<<grid, kThreads, 0, s>>>(static_cast<const T*>(x), static_cast<const T*>(dy), w, mean, rstd,
                                                     static_cast<T*>(dx), rows, width);
    layernorm_dw_kernel<T><<<dim3((unsigned)((width + kThreads - 1) / kThreads), part_rows(rows)), kThreads, 0, s>>>(
        static_cast<const T*>(x), static_cast<const T*>(dy), mean, rstd, part, rows, width);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_layernorm_fwd(long long rows, long long width, int dtype, float eps, const void* x,
                                        const float* weight, const float* bias, void* y, float* mean, float* rstd,
                                        void* stream) {
    if (!valid_size(rows, width)) return KDA_ERR_SHAPE;
    if (dtype != KDA_BF16 && dtype != KDA_FP32) return KDA_ERR_UNSUPPORTED;
    if (!(std::isfinite(eps) && eps > 0.0f)) return KDA_ERR_UNSUPPORTED;
    if (rows == 0) return KDA_OK;
    if (!x || !y) return KDA_ERR_NULL;
    const void* ptrs[] = {x, weight, bias, y, mean, rstd};
    for (const void* p : ptrs)
        if (misaligned(p)) return KDA_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == KDA_BF16) fwd<uint16_t>(rows, (int)width, eps, x, weight, bias, y, mean, rstd, s);
    else fwd<float>(rows, (int)width, eps, x, weight, bias, y, mean, rstd, s);
    return launched("kda_layernorm_fwd launch");
}

extern "C" size_t kda_layernorm_workspace_size(long long rows, long long width) {
    if (!valid_size(rows, width)) return 0;
    return align_up((size_t)kPartRows * 2 * (size_t)width * sizeof(float), 1024);
}

extern "C" kda_status kda_layernorm_bwd(long long rows, long long width, int dtype, const void* x, const void* dy,
                                        const float* weight, const float* mean, const float* rstd, void* dx,
                                        float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                                        void* stream) {
    if (!valid_size(rows, width)) return KDA_ERR_SHAPE;
    if (dtype != KDA_BF16 && dtype != KDA_FP32) return KDA_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < kda_layernorm_workspace_size(rows, width)) return KDA_ERR_WORKSPACE;
    if (rows > 0 && (!x || !dy || !mean || !rstd || !dx)) return KDA_ERR_NULL;
    const void* ptrs[] = {x, dy, weight, mean, rstd, dx, dweight, dbias, workspace};
    for (const void* p : ptrs)
        if (misaligned(p)) return KDA_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    float* part = static_cast<float*>(workspace);
    if (rows > 0) {
        if (dtype == KDA_BF16) bwd<uint16_t>(rows, (int)width, x, dy, weight, mean, rstd, dx, part, s);
        else bwd<float>(rows, (int)width, x, dy, weight, mean, rstd, dx, part, s);
    }
    if (dweight || dbias)
        layernorm_reduce_kernel<<<(unsigned)((width + kThreads - 1) / kThreads), kThreads, 0, s>>>(
            part, (int)part_rows(rows), (int)width, dweight, dbias);
    return launched("kda_layernorm_bwd launch");
}
