// Gated recurrence over channels, forward, backward and single tokens.
//   u = exp(A_log) s, s = sigmoid(g_raw), a = exp(-u), m = sqrt(1 - a^2), i = sigmoid(i_raw)
//   h_t = a_t h_{t-1} + m_t i_t x_t
//   G_t = dy_t + a_{t+1} G_{t+1}   (dhT in place of the second after a sequence's last token)
//   dx = G m i,  di_raw = G m x i (1 - i),  dh0 = a G at the first token
//   du u = G (i x a^2 u / m - u a h_{t-1}),  dg_raw = du u (1 - s),  dA_log = sum du u
// em = 1 - a is what the arithmetic holds: -expm1(-u), a series for small u, so that h += b - em h keeps
// fp32's precision over memories of any length, and m = sqrt(em (2 - em)) has no cancellation.
// Simple form: a thread takes a channel of a sequence, token after token.
#include <cmath>
#include <cstdio>
#include "kda_internal.cuh"

namespace kda {
void set_last_error_text(const char* msg);

namespace {
constexpr int kBlock = KDA_RECURRENCE_BLOCK;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float get(const uint16_t* p) { return bf2f(*p); }
__device__ __forceinline__ float get(const float* p) { return *p; }
__device__ __forceinline__ void put(uint16_t* p, float x) { *p = f2bf(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }

// sigmoid(x) and 1 - sigmoid(x), without cancellation at either end
struct Sigmoid {
    float s, c;
};
__device__ __forceinline__ Sigmoid sigmoid2(float x) {
    const float e = exp2f(fminf(-x * kLog2e, 126.0f));   // finite, so that e * s is
    const float s = 1.0f / (1.0f + e);
    return {s, e * s};
}

// 1 - exp(-u) for u >= 0: below 1/4 the series u - u^2/2 + u^3/6 .. u^6/720 (the next term is 5e-8 of the sum), above
// it 1 - exp(-u), which loses two bits at most there
__device__ __forceinline__ float one_minus_exp(float u) {
    const float p = u * (1.0f + u * (-1.0f / 2 + u * (1.0f / 6 + u * (-1.0f / 24 + u * (1.0f / 120 + u * (-1.0f / 720))))));
    return u < 0.25f ? p : 1.0f - exp2f(-u * kLog2e);
}

// [first, last) of sequence n, within the tokens whatever the offsets hold
__device__ __forceinline__ void range_of(const int64_t* cu, int64_t T, int64_t total, int64_t n, int64_t& first, int64_t& last) {
    first = cu ? cu[n] : n * T;
    last = cu ? cu[n + 1] : (n + 1) * T;
    first = first < 0 ? 0 : first > total ? total : first;
    last = last < first ? first : last > total ? total : last;
}

// the first block checks the offsets and writes the status word
__device__ __forceinline__ void check_offsets(const int64_t* cu, int64_t N, int64_t total, uint8_t* ws) {
    int bad = 0;
    if (cu) {
        for (int64_t n = threadIdx.x; n < N; n += blockDim.x) bad |= cu[n] > cu[n + 1];
        bad |= cu[0] != 0 || cu[N] != total;
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *reinterpret_cast<int*>(ws) = bad ? KDA_ERR_OFFSETS : KDA_OK;
}

struct RecArgs {
    const void *x, *g, *i, *dy;
    const float *A_log, *h0, *dhT;
    const int64_t* cu;
    void *y, *dx, *dg, *di;
    float *hT, *kept, *dh0, *part;
    uint8_t* ws;
    int64_t total, T, D, N, sx, sg, si, sy, sdx, sdg, sdi;
};

template <typename T> __global__ void __launch_bounds__(128) rec_fwd_kernel(const RecArgs a) {
    if (blockIdx.x == 0) check_offsets(a.cu, a.N, a.total, a.ws);
    const int64_t tiles = (a.D + 127) / 128, c = (blockIdx.x % tiles) * 128 + threadIdx.x, n = blockIdx.x / tiles;
    if (c >= a.D) return;
    int64_t first, last;
    range_of(a.cu, a.T, a.total, n, first, last);
    float h = a.h0 ? a.h0[n * a.D + c] : 0.0f;
    const float lam = expf(a.A_log[c]);
    if (a.kept && first == 0 && last > 0) a.kept[c] = 0.0f;
    for (int64_t t = first; t < last; ++t) {
        const Sigmoid s = sigmoid2(get(static_cast<const T*>(a.g) + t * a.sg + c));
        const Sigmoid i = sigmoid2(get(static_cast<const T*>(a.i) + t * a.si + c));
        const float em = one_minus_exp(lam * s.s);
        const float b = sqrtf(em * (2.0f - em)) * i.s * get(static_cast<const T*>(a.x) + t * a.sx + c);
        h += b - em * h;
        put(static_cast<T*>(a.y) + t * a.sy + c, h);
        if (a.kept && (t + 1) % kBlock == 0 && t + 1 < a.total) a.kept[(t + 1) / kBlock * a.D + c] = h;
    }
    if (a.hT) a.hT[n * a.D + c] = h;
}

template <typename T> __global__ void __launch_bounds__(128) rec_bwd_kernel(const RecArgs a) {
    if (blockIdx.x == 0) check_offsets(a.cu, a.N, a.total, a.ws);
    const int64_t tiles = (a.D + 127) / 128, c = (blockIdx.x % tiles) * 128 + threadIdx.x, n = blockIdx.x / tiles;
    if (c >= a.D) return;
    int64_t first, last;
    range_of(a.cu, a.T, a.total, n, first, last);
    const float lam = expf(a.A_log[c]);
    float acc = 0.0f, G = a.dhT ? a.dhT[n * a.D + c] : 0.0f;
    float before[kBlock];
    for (int64_t j = (last - 1) / kBlock; last > first && j >= first / kBlock; --j) {
        const int64_t t0 = j * kBlock > first ? j * kBlock : first, t1 = (j + 1) * kBlock < last ? (j + 1) * kBlock : last;
        float h = t0 == first ? (a.h0 ? a.h0[n * a.D + c] : 0.0f) : a.kept[j * a.D + c];
        for (int64_t t = t0; t < t1; ++t) {
            before[t - t0] = h;
            const float em = one_minus_exp(lam * sigmoid2(get(static_cast<const T*>(a.g) + t * a.sg + c)).s);
            const float i = sigmoid2(get(static_cast<const T*>(a.i) + t * a.si + c)).s;
            h += sqrtf(em * (2.0f - em)) * i * get(static_cast<const T*>(a.x) + t * a.sx + c) - em * h;
        }
        for (int64_t t = t1 - 1; t >= t0; --t) {
            const Sigmoid s = sigmoid2(get(static_cast<const T*>(a.g) + t * a.sg + c));
            const Sigmoid i = sigmoid2(get(static_cast<const T*>(a.i) + t * a.si + c));
            const float x = get(static_cast<const T*>(a.x) + t * a.sx + c);
            const float u = lam * s.s, em = one_minus_exp(u), m2 = em * (2.0f - em), m = sqrtf(m2), d = 1.0f - em;
            G += get(static_cast<const T*>(a.dy) + t * a.sy + c);
            const float duu = G * (i.s * x * d * d * (m > 0.0f ? u / m : 0.0f) - u * d * before[t - t0]);
            acc += duu;
            put(static_cast<T*>(a.dx) + t * a.sdx + c, G * m * i.s);
            put(static_cast<T*>(a.dg) + t * a.sdg + c, duu * s.c);
            put(static_cast<T*>(a.di) + t * a.sdi + c, G * m * x * i.s * i.c);
            G -= em * G;
        }
    }
    if (a.dh0) a.dh0[n * a.D + c] = G;
    if (a.part) a.part[n * a.D + c] = acc;
}

__global__ void __launch_bounds__(128) rec_sum_kernel(const float* part, int64_t parts, int64_t D, float* out) {
    const int64_t c = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (c >= D) return;
    float s = 0.0f;
    for (int64_t p = 0; p < parts; ++p) s += part[p * D + c];
    out[c] = s;
}

template <typename T> __global__ void __launch_bounds__(256) rec_decode_kernel(const RecArgs a) {
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at >= a.N * a.D) return;
    const int64_t t = at / a.D, c = at % a.D;
    const float em = one_minus_exp(expf(a.A_log[c]) * sigmoid2(get(static_cast<const T*>(a.g) + t * a.sg + c)).s);
    const float b = sqrtf(em * (2.0f - em)) * sigmoid2(get(static_cast<const T*>(a.i) + t * a.si + c)).s *
                    get(static_cast<const T*>(a.x) + t * a.sx + c);
    float h = a.hT[at];
    h += b - em * h;
    a.hT[at] = h;
    put(static_cast<T*>(a.y) + t * a.sy + c, h);
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

kda_status check_shape(const kda_recurrence_shape* sh, bool packed) {
    if (!sh) return KDA_ERR_NULL;
    if (sh->dtype != KDA_BF16 && sh->dtype != KDA_FP32) return KDA_ERR_UNSUPPORTED;
    if (sh->B < 0 || sh->T < 0 || sh->N < 0 || sh->D <= 0 || sh->D > (1 << 20)) return KDA_ERR_SHAPE;
    if (packed ? sh->B != 1 : sh->N != sh->B) return KDA_ERR_SHAPE;
    const int64_t most = (int64_t(1) << 31) - 1;
    if (sh->B > most || sh->T > most || sh->N > most || (sh->T > 0 && sh->B > most / sh->T)) return KDA_ERR_SHAPE;
    if (sh->B * sh->T > 0 && sh->N == 0) return KDA_ERR_SHAPE;
    const int64_t strides[] = {sh->x_stride, sh->g_stride, sh->i_stride, sh->y_stride, sh->dx_stride, sh->dg_stride, sh->di_stride};
    for (const int64_t s : strides)
        if (s != 0 && (s < sh->D || s > (int64_t(1) << 40))) return KDA_ERR_SHAPE;
    return KDA_OK;
}

size_t bytes_of(const kda_recurrence_shape* sh, bool backward) {
    return 1024 + (backward ? align_up((size_t)sh->N * sh->D * sizeof(float), 1024) : 0);
}

RecArgs args_of(const kda_recurrence_shape* sh) {
    RecArgs a{};
    auto st = [&](int64_t s) { return s ? s : sh->D; };
    a.total = sh->B * sh->T; a.T = sh->T; a.D = sh->D; a.N = sh->N;
    a.sx = st(sh->x_stride); a.sg = st(sh->g_stride); a.si = st(sh->i_stride); a.sy = st(sh->y_stride);
    a.sdx = st(sh->dx_stride); a.sdg = st(sh->dg_stride); a.sdi = st(sh->di_stride);
    return a;
}

kda_status common_checks(const kda_recurrence_shape* sh, const int64_t* cu, const void* ws, size_t bytes, bool backward) {
    const kda_status st = check_shape(sh, cu != nullptr);
    if (st != KDA_OK) return st;
    if (!ws || bytes < bytes_of(sh, backward)) return KDA_ERR_WORKSPACE;
    if (misaligned(ws) || misaligned(cu, 8)) return KDA_ERR_ALIGN;
    return KDA_OK;
}
}  // namespace
}  // namespace kda

using namespace kda;

extern "C" size_t kda_recurrence_workspace_size(const kda_recurrence_shape* shape, int backward) {
    if (!shape || (check_shape(shape, true) != KDA_OK && check_shape(shape, false) != KDA_OK)) return 0;
    return bytes_of(shape, backward != 0);
}

extern "C" kda_status kda_recurrence_fwd(const kda_recurrence_shape* shape, const void* x, const void* g_raw, const void* i_raw,
                                         const float* A_log, const float* h0, const int64_t* cu_seqlens, void* y, float* hT,
                                         float* kept, void* workspace, size_t workspace_bytes, void* stream) {
    const kda_status st = common_checks(shape, cu_seqlens, workspace, workspace_bytes, false);
    if (st != KDA_OK) return st;
    if (!A_log || (shape->B * shape->T > 0 && (!x || !g_raw || !i_raw || !y))) return KDA_ERR_NULL;
    const uintptr_t e = shape->dtype == KDA_BF16 ? 2 : 4;
    for (const void* p : {x, g_raw, i_raw, static_cast<const void*>(y)})
        if (misaligned(p, e)) return KDA_ERR_ALIGN;
    for (const float* p : {A_log, h0, static_cast<const float*>(hT), static_cast<const float*>(kept)})
        if (misaligned(p)) return KDA_ERR_ALIGN;
    if (hT && hT == h0) return KDA_ERR_UNSUPPORTED;
    if (shape->N == 0) return KDA_OK;
    RecArgs a = args_of(shape);
    a.x = x; a.g = g_raw; a.i = i_raw; a.y = y; a.A_log = A_log; a.h0 = h0; a.cu = cu_seqlens; a.hT = hT; a.kept = kept;
    a.ws = static_cast<uint8_t*>(workspace);
    const int64_t blocks = (a.D + 127) / 128 * a.N;
    if (blocks >= (int64_t(1) << 31)) return KDA_ERR_SHAPE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (shape->dtype == KDA_BF16) rec_fwd_kernel<uint16_t><<<(unsigned)blocks, 128, 0, s>>>(a);
    else rec_fwd_kernel<float><<<(unsigned)blocks, 128, 0, s>>>(a);
    return launched("kda_recurrence_fwd launch");
}

extern "C" kda_status kda_recurrence_bwd(const kda_recurrence_shape* shape, const void* x, const void* g_raw, const void* i_raw,
                                         const float* A_log, const float* h0, const int64_t* cu_seqlens, const void* dy,
                                         const float* dhT, const float* kept, void* dx, void* dg_raw, void* di_raw,
                                         float* dA_log, float* dh0, void* workspace, size_t workspace_bytes, void* stream) {
    const kda_status st = common_checks(shape, cu_seqlens, workspace, workspace_bytes, true);
    if (st != KDA_OK) return st;
    const bool some = shape->B * shape->T > 0;
    if (!A_log || (some && (!x || !g_raw || !i_raw || !dy || !kept || !dx || !dg_raw || !di_raw))) return KDA_ERR_NULL;
    const uintptr_t e = shape->dtype == KDA_BF16 ? 2 : 4;
    for (const void* p : {x, g_raw, i_raw, dy, static_cast<const void*>(dx), static_cast<const void*>(dg_raw), static_cast<const void*>(di_raw)})
        if (misaligned(p, e)) return KDA_ERR_ALIGN;
    for (const float* p : {A_log, h0, dhT, kept, static_cast<const float*>(dA_log), static_cast<const float*>(dh0)})
        if (misaligned(p)) return KDA_ERR_ALIGN;
    if (dh0 && dh0 == dhT) return KDA_ERR_UNSUPPORTED;
    RecArgs a = args_of(shape);
    a.x = x; a.g = g_raw; a.i = i_raw; a.dy = dy; a.A_log = A_log; a.h0 = h0; a.dhT = dhT; a.cu = cu_seqlens;
    a.kept = const_cast<float*>(kept); a.dx = dx; a.dg = dg_raw; a.di = di_raw; a.dh0 = dh0;
    a.ws = static_cast<uint8_t*>(workspace);
    a.part = reinterpret_cast<float*>(a.ws + 1024);
    const int64_t blocks = (a.D + 127) / 128 * a.N;
    if (blocks >= (int64_t(1) << 31)) return KDA_ERR_SHAPE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (blocks > 0) {
        if (shape->dtype == KDA_BF16) rec_bwd_kernel<uint16_t><<<(unsigned)blocks, 128, 0, s>>>(a);
        else rec_bwd_kernel<float><<<(unsigned)blocks, 128, 0, s>>>(a);
    }
    if (dA_log) rec_sum_kernel<<<(unsigned)((a.D + 127) / 128), 128, 0, s>>>(a.part, a.N, a.D, dA_log);
    return launched("kda_recurrence_bwd launch");
}

extern "C" kda_status kda_recurrence_decode(const kda_recurrence_shape* shape, const void* x, const void* g_raw,
                                            const void* i_raw, const float* A_log, float* state, void* y, void* stream) {
    const kda_status st = check_shape(shape, false);
    if (st != KDA_OK) return st;
    if (shape->T != 1) return KDA_ERR_SHAPE;
    if (shape->N == 0) return KDA_OK;
    if (!x || !g_raw || !i_raw || !A_log || !state || !y) return KDA_ERR_NULL;
    const uintptr_t e = shape->dtype == KDA_BF16 ? 2 : 4;
    for (const void* p : {x, g_raw, i_raw, static_cast<const void*>(y)})
        if (misaligned(p, e)) return KDA_ERR_ALIGN;
    if (misaligned(A_log) || misaligned(state)) return KDA_ERR_ALIGN;
    RecArgs a = args_of(shape);
    a.x = x; a.g = g_raw; a.i = i_raw; a.A_log = A_log; a.hT = state; a.y = y;
    const int64_t blocks = (a.N * a.D + 255) / 256;
    if (blocks >= (int64_t(1) << 31)) return KDA_ERR_SHAPE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (shape->dtype == KDA_BF16) rec_decode_kernel<uint16_t><<<(unsigned)blocks, 256, 0, s>>>(a);
    else rec_decode_kernel<float><<<(unsigned)blocks, 256, 0, s>>>(a);
    return launched("kda_recurrence_decode launch");
}
