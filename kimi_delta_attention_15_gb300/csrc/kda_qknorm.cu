// Norm of queries and keys by heads with the position rotation in the same pass, forward and backward.
//   r = 1 / sqrt(mean(x^2) + eps),  z = x r w,  y = z turned by position * inv_freq in pairs
//   gz = dy turned back,  dw = sum gz x r,  dx = r (gz w - x r^2 mean(gz w x))
// A few operations per byte: HBM is the floor. A lane holds 8 columns of a row in registers, the two sides of four
// pairs, so that a rotation needs no exchange: columns 4 p .. 4 p + 3 and rotary/2 + 4 p .. of unit p where pairs are half of
// the rotated columns apart, 8 p .. 8 p + 7 elsewhere; only the row's sums go through shuffles. A warp takes a
// token (or a share of its heads, where tokens are few), so that sines and cosines are computed once for many heads.
// An angle is a fraction of a turn in 64-bit fixed point: inv_freq / 2 pi comes from its 24 bits and a 128-bit
// constant, and position times that, modulo 2^64, is exact at any position.
#include <cmath>
#include <cstdio>
#include "kda_internal.cuh"
#include "umma_bf16.cuh"

namespace kda {
void set_last_error_text(const char* msg);

namespace {
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSMs = 152;
constexpr int kRows = 4;         // rows of a lane in flight
constexpr int kBlocksPerSM = 4;

// inv_freq / 2 pi as a 64-bit fraction of a turn, truncated at 2^-64: the significand times 1 / 2 pi in 128 bits, shifted
__device__ __forceinline__ uint64_t turn_fraction(float f) {
    const uint32_t bits = __float_as_uint(f), field = (bits >> 23) & 255u;
    const uint64_t mant = (bits & 0x7fffffu) | (field ? 0x800000u : 0u);
    const int shift = 64 - ((field ? (int)field : 1) - 150);
    constexpr uint64_t kHi = 0x28be60db9391054aull, kLo = 0x7f09d5f47d4d3770ull;   // 2^128 / 2 pi
    const uint64_t lo = mant * kLo, carry = __umul64hi(mant, kLo), mid = mant * kHi + carry;
    const uint64_t hi = __umul64hi(mant, kHi) + (mid < carry ? 1u : 0u);
    uint64_t r;
    if (shift <= 0) r = shift > -64 ? lo << -shift : 0;
    else if (shift < 64) r = (lo >> shift) | (mid << (64 - shift));
    else if (shift == 64) r = mid;
    else if (shift < 128) r = (mid >> (shift - 64)) | (hi << (128 - shift));
    else r = shift < 192 ? hi >> (shift - 128) : 0;
    return bits >> 31 ? 0 - r : r;
}

// four consecutive columns
__device__ __forceinline__ void load4(const uint16_t* p, float* v) {
    const uint2 w = __ldcs(reinterpret_cast<const uint2*>(p));
    v[0] = __uint_as_float(w.x << 16); v[1] = __uint_as_float(w.x & 0xffff0000u);
    v[2] = __uint_as_float(w.y << 16); v[3] = __uint_as_float(w.y & 0xffff0000u);
}
__device__ __forceinline__ void load4(const float* p, float* v) {
    const float4 w = __ldcs(reinterpret_cast<const float4*>(p));
    v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
}
__device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store4(uint16_t* p, const float* v) {
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(pack(v[0], v[1]), pack(v[2], v[3])));
}
__device__ __forceinline__ void store4(float* p, const float* v) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
}

struct Side {            // q or k
    const void *x, *dy;
    void* out;           // y, or dx in the backward
    const float* w;
    int64_t sx, sdy, sout;
    int heads, blocks;   // blocks of kRows rows of each group of lanes
};
struct QkArgs {
    Side side[2];
    const int64_t* positions;
    const float* inv_freq;
    float* part;         // [blocks of the grid][2][head] sums of the weights' gradients, or NULL
    int64_t tokens;
    int head, rotary, lanes, splits;   // lanes: of a row, a power of two
    float eps, inv_head;
};

// What a lane keeps between tokens
struct Lane {
    int unit, group, groups, c1, c2;
    bool on, turned;
    uint64_t f[4];
    __device__ __forceinline__ Lane(const QkArgs& a, bool interleaved) {
        const int lane = threadIdx.x & 31;
        unit = lane & (a.lanes - 1);
        group = lane / a.lanes;
        groups = 32 / a.lanes;
        on = 8 * unit < a.head;
        turned = 8 * unit < a.rotary;
        const bool half = turned && !interleaved;
        c1 = half ? 4 * unit : 8 * unit;
        c2 = half ? a.rotary / 2 + 4 * unit : 8 * unit + 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = turned ? turn_fraction(a.inv_freq[4 * unit + j]) : 0;
    }
    __device__ __forceinline__ void weights(const float* w, float* v) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = w && on ? w[c1 + j] : 1.0f;
            v[4 + j] = w && on ? w[c2 + j] : 1.0f;
        }
    }
    __device__ __forceinline__ void angles(int64_t position, float* cs, float* sn) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int32_t top = (int32_t)((f[j] * (uint64_t)position) >> 32);   // of a turn, from -1/2 to 1/2
            sincospif((float)top * 0x1p-31f, &sn[j], &cs[j]);
        }
    }
};

template <bool kInterleaved> __device__ __forceinline__ void turn(float* v, const float* cs, const float* sn) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float &a = v[kInterleaved ? 2 * j : j], &b = v[kInterleaved ? 2 * j + 1 : 4 + j];
        const float x = a * cs[j] - b * sn[j];
        b = b * cs[j] + a * sn[j];
        a = x;
    }
}

template <typename T, bool kInterleaved> __global__ void __launch_bounds__(kThreads) qknorm_fwd_kernel(const QkArgs a) {
    const Lane l(a, kInterleaved);
    float w[2][8];
    l.weights(a.side[0].w, w[0]);
    l.weights(a.side[1].w, w[1]);
    const int64_t items = a.tokens * a.splits, step = (int64_t)gridDim.x * kWarps;
    for (int64_t it = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); it < items; it += step) {
        const int64_t t = it / a.splits;
        float cs[4], sn[4];
        l.angles(a.rotary ? a.positions[t] : 0, cs, sn);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const Side& s = a.side[k];
            const int first = (int)(it % a.splits) - (k ? a.side[0].blocks : 0);
            for (int b = first < 0 ? first + (-first + a.splits - 1) / a.splits * a.splits : first; b < s.blocks; b += a.splits) {
                float v[kRows][8];
                const int h0 = b * kRows * l.groups + l.group;
                const T* x = static_cast<const T*>(s.x) + t * s.sx;
                T* y = static_cast<T*>(s.out) + t * s.sout;
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    const int h = h0 + i * l.groups;
                    if (l.on && h < s.heads) {
                        load4(x + h * a.head + l.c1, v[i]);
                        load4(x + h * a.head + l.c2, v[i] + 4);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
                    }
                }
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    float ss = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) ss += v[i][j] * v[i][j];
                    for (int o = a.lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    const float r = rsqrtf(ss * a.inv_head + a.eps);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i][j] *= r * w[k][j];
                    turn<kInterleaved>(v[i], cs, sn);
                    const int h = h0 + i * l.groups;
                    if (l.on && h < s.heads) {
                        store4(y + h * a.head + l.c1, v[i]);
                        store4(y + h * a.head + l.c2, v[i] + 4);
                    }
                }
            }
        }
    }
}

template <typename T, bool kInterleaved> __global__ void __launch_bounds__(kThreads) qknorm_bwd_kernel(const QkArgs a) {
    const Lane l(a, kInterleaved);
    float w[2][8], dw[2][8];
    l.weights(a.side[0].w, w[0]);
    l.weights(a.side[1].w, w[1]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[0][j] = dw[1][j] = 0.0f;
    const int64_t items = a.tokens * a.splits, step = (int64_t)gridDim.x * kWarps;
    for (int64_t it = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); it < items; it += step) {
        const int64_t t = it / a.splits;
        float cs[4], sn[4];
        l.angles(a.rotary ? -a.positions[t] : 0, cs, sn);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const Side& s = a.side[k];
            const int first = (int)(it % a.splits) - (k ? a.side[0].blocks : 0);
            for (int b = first < 0 ? first + (-first + a.splits - 1) / a.splits * a.splits : first; b < s.blocks; b += a.splits) {
                const int h0 = b * kRows * l.groups + l.group;
                const T* x = static_cast<const T*>(s.x) + t * s.sx;
                const T* dy = static_cast<const T*>(s.dy) + t * s.sdy;
                T* dx = static_cast<T*>(s.out) + t * s.sout;
                float v[kRows][8], g[kRows][8];
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    const int h = h0 + i * l.groups;
                    if (l.on && h < s.heads) {
                        load4(x + h * a.head + l.c1, v[i]);
                        load4(x + h * a.head + l.c2, v[i] + 4);
                        load4(dy + h * a.head + l.c1, g[i]);
                        load4(dy + h * a.head + l.c2, g[i] + 4);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[i][j] = g[i][j] = 0.0f;
                    }
                }
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    turn<kInterleaved>(g[i], cs, sn);
                    float ss = 0.0f, dot = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        ss += v[i][j] * v[i][j];
                        dot += g[i][j] * w[k][j] * v[i][j];
                    }
                    for (int o = a.lanes >> 1; o > 0; o >>= 1) {
                        ss += __shfl_xor_sync(0xffffffffu, ss, o);
                        dot += __shfl_xor_sync(0xffffffffu, dot, o);
                    }
                    const float r = rsqrtf(ss * a.inv_head + a.eps), m = dot * a.inv_head * r * r;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        dw[k][j] += g[i][j] * (v[i][j] * r);
                        g[i][j] = r * (g[i][j] * w[k][j] - v[i][j] * m);
                    }
                    const int h = h0 + i * l.groups;
                    if (l.on && h < s.heads) {
                        store4(dx + h * a.head + l.c1, g[i]);
                        store4(dx + h * a.head + l.c2, g[i] + 4);
                    }
                }
            }
        }
    }
    if (!a.part) return;
    grid_launch_next();
    // a block's sums: the groups of a warp, then the warps in turn
    __shared__ float sums[kWarps][2][256];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            for (int o = 16; o >= a.lanes; o >>= 1) dw[k][j] += __shfl_xor_sync(0xffffffffu, dw[k][j], o);
            if (l.group == 0 && l.on) sums[threadIdx.x >> 5][k][(j < 4 ? l.c1 : l.c2) + (j & 3)] = dw[k][j];
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.head; i += kThreads) {
        const int k = i >= a.head, c = i - k * a.head;
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < kWarps; ++v) s += sums[v][k][c];
        a.part[((int64_t)blockIdx.x * 2 + k) * a.head + c] = s;
    }
}

// The sums over blocks, 32 columns by 32 threads each, in a fixed order.
__global__ void __launch_bounds__(1024) qknorm_sum_kernel(const float* part, int parts, int head, float* dq, float* dk) {
    grid_wait_before();
    __shared__ float sums[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x, k = blockIdx.y;
    float* const out = k ? dk : dq;
    if (!out) return;
    float s = 0.0f;
    if (c < head)
        for (int p = threadIdx.y; p < parts; p += 32) s += part[((int64_t)p * 2 + k) * head + c];
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < head) {
        s = 0.0f;
        for (int i = 0; i < 32; ++i) s += sums[i][threadIdx.x];
        out[c] = s;
    }
}

bool misaligned(const void* p, uintptr_t to = 16) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

kda_status launched(const char* where) {
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return KDA_OK;
    char msg[160];
    snprintf(msg, sizeof(msg), "%s: %s (%d)", where, cudaGetErrorString(e), (int)e);
    set_last_error_text(msg);
    return KDA_ERR_CUDA;
}

constexpr int64_t kMostStride = int64_t(1) << 40;

kda_status check_shape(const kda_qknorm_shape* sh) {
    if (!sh) return KDA_ERR_NULL;
    if (sh->dtype != KDA_BF16 && sh->dtype != KDA_FP32) return KDA_ERR_UNSUPPORTED;
    if (!(std::isfinite(sh->eps) && sh->eps > 0.0f)) return KDA_ERR_UNSUPPORTED;
    if (sh->interleaved != 0 && sh->interleaved != 1) return KDA_ERR_UNSUPPORTED;
    if (sh->tokens < 0 || sh->tokens >= (int64_t(1) << 31) || sh->q_heads <= 0 || sh->q_heads > (1 << 20) || sh->k_heads < 0 ||
        sh->k_heads > (1 << 20))
        return KDA_ERR_SHAPE;
    if (sh->head_dim <= 0 || sh->head_dim > 256 || sh->head_dim % 8) return KDA_ERR_UNSUPPORTED;
    if (sh->rotary_dim < 0 || sh->rotary_dim > sh->head_dim || sh->rotary_dim % 8) return KDA_ERR_UNSUPPORTED;
    const int64_t q = (int64_t)sh->q_heads * sh->head_dim, k = (int64_t)sh->k_heads * sh->head_dim;
    for (const int64_t s : {sh->q_stride, sh->q_out_stride, sh->dq_stride})
        if (s && (s < q || s > kMostStride)) return KDA_ERR_SHAPE;
    for (const int64_t s : {sh->k_stride, sh->k_out_stride, sh->dk_stride})
        if (s && (s < k || s > kMostStride)) return KDA_ERR_SHAPE;
    const int unit = sh->dtype == KDA_BF16 ? 8 : 4;
    for (const int64_t s : {sh->q_stride, sh->q_out_stride, sh->dq_stride, sh->k_stride, sh->k_out_stride, sh->dk_stride})
        if (s % unit) return KDA_ERR_ALIGN;
    return KDA_OK;
}

int64_t or_else(int64_t stride, int64_t width) { return stride ? stride : width; }

QkArgs args_of(const kda_qknorm_shape* sh) {
    QkArgs a{};
    a.tokens = sh->tokens;
    a.head = sh->head_dim;
    a.rotary = sh->rotary_dim;
    a.eps = sh->eps;
    a.inv_head = 1.0f / sh->head_dim;
    a.lanes = 1;
    while (8 * a.lanes < a.head) a.lanes *= 2;
    const int rows = kRows * (32 / a.lanes);
    a.side[0].heads = sh->q_heads;
    a.side[1].heads = sh->k_heads;
    for (Side& s : a.side) s.blocks = (s.heads + rows - 1) / rows;
    // a warp for each token while these fill the GPU, else several to share a token's heads
    const int64_t want = (int64_t)kSMs * kBlocksPerSM * kWarps, most = a.side[0].blocks + a.side[1].blocks;
    const int64_t n = sh->tokens ? (want + sh->tokens - 1) / sh->tokens : 1;
    a.splits = (int)(n < most ? n : most);
    return a;
}
unsigned grid_of(const QkArgs& a) {
    const int64_t blocks = (a.tokens * a.splits + kWarps - 1) / kWarps, most = (int64_t)kSMs * kBlocksPerSM;
    return (unsigned)(blocks < most ? blocks : most);
}
}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_qknorm_fwd(const kda_qknorm_shape* shape, const void* q, const void* k, const float* q_weight,
                                     const float* k_weight, const int64_t* positions, const float* inv_freq, void* q_out,
                                     void* k_out, void* stream) {
    const kda_status st = check_shape(shape);
    if (st != KDA_OK) return st;
    if (shape->tokens == 0) return KDA_OK;
    const bool keys = shape->k_heads > 0, turned = shape->rotary_dim > 0;
    if (!q || !q_out || (keys && (!k || !k_out)) || (turned && (!positions || !inv_freq))) return KDA_ERR_NULL;
    for (const void* p : {q, static_cast<const void*>(q_out), static_cast<const void*>(q_weight), static_cast<const void*>(inv_freq)})
        if (misaligned(p)) return KDA_ERR_ALIGN;
    for (const void* p : {k, static_cast<const void*>(k_out), static_cast<const void*>(k_weight)})
        if (keys && misaligned(p)) return KDA_ERR_ALIGN;
    if (misaligned(positions, 8)) return KDA_ERR_ALIGN;
    QkArgs a = args_of(shape);
    const int64_t wq = (int64_t)shape->q_heads * shape->head_dim, wk = (int64_t)shape->k_heads * shape->head_dim;
    a.side[0] = Side{q, nullptr, q_out, q_weight, or_else(shape->q_stride, wq), 0, or_else(shape->q_out_stride, wq), a.side[0].heads, a.side[0].blocks};
    a.side[1] = Side{k, nullptr, k_out, keys ? k_weight : nullptr, or_else(shape->k_stride, wk), 0, or_else(shape->k_out_stride, wk), a.side[1].heads, a.side[1].blocks};
    a.positions = positions;
    a.inv_freq = inv_freq;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto run = shape->dtype == KDA_BF16 ? (shape->interleaved ? qknorm_fwd_kernel<uint16_t, true> : qknorm_fwd_kernel<uint16_t, false>)
                                        : (shape->interleaved ? qknorm_fwd_kernel<float, true> : qknorm_fwd_kernel<float, false>);
    run<<<grid_of(a), kThreads, 0, s>>>(a);
    return launched("kda_qknorm_fwd launch");
}

extern "C" size_t kda_qknorm_workspace_size(const kda_qknorm_shape* shape) {
    if (check_shape(shape) != KDA_OK) return 0;
    const QkArgs a = args_of(shape);
    return align_up((size_t)(grid_of(a) + 1) * 2 * a.head * sizeof(float), 1024);
}

extern "C" kda_status kda_qknorm_bwd(const kda_qknorm_shape* shape, const void* q, const void* k, const void* dq_out,
                                     const void* dk_out, const float* q_weight, const float* k_weight,
                                     const int64_t* positions, const float* inv_freq, void* dq, void* dk, float* dq_weight,
                                     float* dk_weight, void* workspace, size_t workspace_bytes, void* stream) {
    const kda_status st = check_shape(shape);
    if (st != KDA_OK) return st;
    if (!workspace || workspace_bytes < kda_qknorm_workspace_size(shape)) return KDA_ERR_WORKSPACE;
    const bool some = shape->tokens > 0, keys = shape->k_heads > 0, turned = shape->rotary_dim > 0;
    if (some && (!q || !dq_out || !dq || (keys && (!k || !dk_out || !dk)) || (turned && (!positions || !inv_freq)))) return KDA_ERR_NULL;
    for (const void* p : {q, dq_out, static_cast<const void*>(dq), static_cast<const void*>(q_weight), static_cast<const void*>(inv_freq),
                          static_cast<const void*>(dq_weight), static_cast<const void*>(dk_weight), static_cast<const void*>(workspace)})
        if (misaligned(p)) return KDA_ERR_ALIGN;
    for (const void* p : {k, dk_out, static_cast<const void*>(dk), static_cast<const void*>(k_weight)})
        if (keys && misaligned(p)) return KDA_ERR_ALIGN;
    if (misaligned(positions, 8)) return KDA_ERR_ALIGN;
    QkArgs a = args_of(shape);
    const int64_t wq = (int64_t)shape->q_heads * shape->head_dim, wk = (int64_t)shape->k_heads * shape->head_dim;
    a.side[0] = Side{q, dq_out, dq, q_weight, or_else(shape->q_stride, wq), or_else(shape->q_out_stride, wq), or_else(shape->dq_stride, wq), a.side[0].heads, a.side[0].blocks};
    a.side[1] = Side{k, dk_out, dk, keys ? k_weight : nullptr, or_else(shape->k_stride, wk), or_else(shape->k_out_stride, wk), or_else(shape->dk_stride, wk), a.side[1].heads, a.side[1].blocks};
    a.positions = positions;
    a.inv_freq = inv_freq;
    const bool sums = dq_weight || dk_weight;
    a.part = sums ? static_cast<float*>(workspace) : nullptr;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned grid = grid_of(a);
    if (grid) {
        auto run = shape->dtype == KDA_BF16 ? (shape->interleaved ? qknorm_bwd_kernel<uint16_t, true> : qknorm_bwd_kernel<uint16_t, false>)
                                            : (shape->interleaved ? qknorm_bwd_kernel<float, true> : qknorm_bwd_kernel<float, false>);
        run<<<grid, kThreads, 0, s>>>(a);
    }
    if (sums)
        launch_kernel(qknorm_sum_kernel, dim3((unsigned)((a.head + 31) / 32), 2), dim3(32, 32), 0, s, grid > 0,
                      static_cast<const float*>(workspace), (int)grid, a.head, dq_weight, dk_weight);
    return launched("kda_qknorm_bwd launch");
}
