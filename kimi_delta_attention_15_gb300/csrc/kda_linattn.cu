// Linear attention with one decay for each head: prompts, their gradient, single tokens.
//   S_t = gamma S_{t-1} + v_t k_t^T,  o_t = scale S_t q_t,  gamma = exp(log_decay[h])
// The gradients are the same sum with other operands:
//   dq_i = scale (sum_{j <= i} gamma^{i-j} (do_i . v_j) k_j + gamma^{i+1} S0^T do_i)
//   dk_j = sum_{i >= j} scale gamma^{i-j} (v_j . do_i) q_i + gamma^{T-1-j} dhT^T v_j
//   dv_j = sum_{i >= j} scale gamma^{i-j} (k_j . q_i) do_i + gamma^{T-1-j} dhT k_j
// so dq is the forward with (q, k, v) <- (do, v, k), and dk, dv are forwards over the
// tokens in reverse with (v, do, q) and (k, q, do). One kernel runs all four as jobs; a
// reversed job differs from a forward one only in the sign of the token stride and in
// whether the decay of a token applies before or after its read:
//   forward   S <- gamma S + v k^T,         out = S q
//   reversed  S <- S + v k^T,  out = S q,   S <- gamma S
#include <cmath>
#include <cstdio>
#include "kda_internal.cuh"

namespace kda {
void set_last_error_text(const char* msg);

namespace {

struct LinJob {
    const uint16_t *q, *k, *v;   // the roles' tensors, [tokens, H / g?, 128]
    int gq, gk, gv;              // value heads that share a head of each
    uint16_t* out;               // [tokens, H, 128] bf16, or
    float* share;                // [tokens, H, 128] fp32: each value head's share of a grouped sum
    const float* s_in;           // initial state [N, H, 128, 128], may be NULL
    float* s_out;                // final state, may be NULL
    int s_in_t;                  // s_in is stored transposed
    int rev;                     // tokens from last to first
    float k_scale, out_scale;    // k is multiplied by the first, the output by the second
};

struct LinArgs {
    LinJob job[3];
    const int64_t* cu;
    const float* log_decay;
    int64_t T;                   // tokens per sequence when fixed
    int H, N;
    uint8_t* ws;
};

// Offsets: cu[0] = 0, non-decreasing, cu[N] = T_total. Starts the status word.
__global__ void __launch_bounds__(1024)
    linattn_offsets_kernel(const int64_t* __restrict__ cu, int64_t N, int64_t T_total, uint8_t* __restrict__ ws) {
    __shared__ int bad;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    if (cu) {
        if (threadIdx.x == 0 && (cu[0] != 0 || cu[N] != T_total)) bad = 1;
        for (int64_t n = threadIdx.x; n < N; n += blockDim.x)
            if (cu[n + 1] < cu[n]) bad = 1;
    }
    __syncthreads();
    if (threadIdx.x == 0) *reinterpret_cast<int*>(ws) = bad ? KDA_ERR_OFFSETS : 0;
}

// One CTA for each (head, sequence, job), token by token: thread v holds row v of the state.
__global__ void __launch_bounds__(128) linattn_kernel(const __grid_constant__ LinArgs a) {
    __shared__ float sq[D], sk[D];
    if (read_status(a.ws) != 0) return;
    const LinJob& jb = a.job[blockIdx.z];
    const int h = blockIdx.x, n = blockIdx.y, v = threadIdx.x;
    const int64_t t0 = a.cu ? a.cu[n] : n * a.T, t1 = a.cu ? a.cu[n + 1] : (n + 1) * a.T;
    const float g = expf(a.log_decay[h]);
    const size_t sidx = ((size_t)n * a.H + h) * D * D;
    float s[D];
#pragma unroll
    for (int c = 0; c < D; ++c) s[c] = jb.s_in ? (jb.s_in_t ? jb.s_in[sidx + c * D + v] : jb.s_in[sidx + v * D + c]) : 0.0f;
    for (int64_t i = 0; i < t1 - t0; ++i) {
        const int64_t t = jb.rev ? t1 - 1 - i : t0 + i;
        __syncthreads();
        sq[v] = bf2f(jb.q[(t * (a.H / jb.gq) + h / jb.gq) * D + v]);
        sk[v] = bf2f(jb.k[(t * (a.H / jb.gk) + h / jb.gk) * D + v]) * jb.k_scale;
        __syncthreads();
        const float vv = bf2f(jb.v[(t * (a.H / jb.gv) + h / jb.gv) * D + v]);
        const float before = jb.rev ? 1.0f : g, after = jb.rev ? g : 1.0f;
        float o = 0.0f;
#pragma unroll
        for (int c = 0; c < D; ++c) {
            s[c] = before * s[c] + vv * sk[c];
            o += s[c] * sq[c];
            s[c] *= after;
        }
        o *= jb.out_scale;
        if (jb.share) jb.share[(t * a.H + h) * D + v] = o;
        else jb.out[(t * a.H + h) * D + v] = f2bf(o);
    }
    if (jb.s_out)
#pragma unroll
        for (int c = 0; c < D; ++c) jb.s_out[sidx + v * D + c] = s[c];
}

// dq, dk of a query/key head: the sum of its G value heads' shares, in head order.
__global__ void __launch_bounds__(256)
    linattn_group_sum_kernel(const float* __restrict__ share_q, const float* __restrict__ share_k, uint16_t* __restrict__ dq,
                             uint16_t* __restrict__ dk, int64_t n4, int G) {
    // n4: groups of 4 channels in dq; the heads of a group are consecutive rows of 128 channels
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n4) return;
    const float4* src = reinterpret_cast<const float4*>(blockIdx.y ? share_k : share_q) + (i >> 5) * G * 32 + (i & 31);
    float4 s = src[0];
    for (int j = 1; j < G; ++j) {
        const float4 x = src[32 * j];
        s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    reinterpret_cast<ushort4*>(blockIdx.y ? dk : dq)[i] = make_ushort4(f2bf(s.x), f2bf(s.y), f2bf(s.z), f2bf(s.w));
}

// One token for each (request, head): the state is read and written once (64 KB each way), so
// the step is bound by HBM. Warp w owns state rows 16 w .. 16 w + 15, lane l key channels
// 4 l .. 4 l + 3 of each, so that a warp moves whole 512-byte rows.
constexpr int kRows = 16;
__global__ void __launch_bounds__(256)
    linattn_decode_kernel(const uint16_t* __restrict__ q, const uint16_t* __restrict__ k, const uint16_t* __restrict__ v,
                          const float* __restrict__ log_decay, float* __restrict__ state, uint16_t* __restrict__ o, int H,
                          int G, float scale) {
    const int64_t unit = blockIdx.x;   // request * H + h
    const int h = (int)(unit % H);
    const size_t qk = ((size_t)(unit / H) * (H / G) + h / G) * D;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c0 = 4 * lane;
    float* S = state + unit * D * D;
    float4 s[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) s[i] = *reinterpret_cast<const float4*>(S + (size_t)(warp * kRows + i) * D + c0);
    const uint2 qw = *reinterpret_cast<const uint2*>(q + qk + c0), kw = *reinterpret_cast<const uint2*>(k + qk + c0);
    const float g = expf(log_decay[h]);
    const float q0 = bf2f((uint16_t)(qw.x & 0xffffu)), q1 = bf2f((uint16_t)(qw.x >> 16));
    const float q2 = bf2f((uint16_t)(qw.y & 0xffffu)), q3 = bf2f((uint16_t)(qw.y >> 16));
    const float k0 = bf2f((uint16_t)(kw.x & 0xffffu)), k1 = bf2f((uint16_t)(kw.x >> 16));
    const float k2 = bf2f((uint16_t)(kw.y & 0xffffu)), k3 = bf2f((uint16_t)(kw.y >> 16));
    float part[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const float vr = bf2f(v[(size_t)unit * D + warp * kRows + i]);
        s[i].x = g * s[i].x + vr * k0; s[i].y = g * s[i].y + vr * k1;
        s[i].z = g * s[i].z + vr * k2; s[i].w = g * s[i].w + vr * k3;
        *reinterpret_cast<float4*>(S + (size_t)(warp * kRows + i) * D + c0) = s[i];
        part[i] = s[i].x * q0 + s[i].y * q1 + s[i].z * q2 + s[i].w * q3;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < kRows; ++i) part[i] += __shfl_xor_sync(0xffffffffu, part[i], d);
    if (lane < kRows) {
        float ov = part[0];
#pragma unroll
        for (int i = 1; i < kRows; ++i) ov = lane == i ? part[i] : ov;
        o[(size_t)unit * D + warp * kRows + lane] = f2bf(scale * ov);
    }
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

int groups_of(const kda_linattn_shape* sh) { return sh->groups > 1 ? sh->groups : 1; }

kda_status check_shape(const kda_linattn_shape* sh, bool packed) {
    if (!sh) return KDA_ERR_NULL;
    if (sh->K != 128 || sh->V != 128) return KDA_ERR_UNSUPPORTED;
    if (!(std::isfinite(sh->scale) && sh->scale > 0.0f)) return KDA_ERR_UNSUPPORTED;
    if (sh->B < 1 || sh->T < 0 || sh->H < 1 || sh->H > 65535 || sh->N < 0) return KDA_ERR_SHAPE;
    if (packed) {
        if (sh->B != 1 || sh->N < 1 || sh->N > 65535) return KDA_ERR_SHAPE;
    } else if (sh->N != sh->B || sh->B > 65535) {
        return KDA_ERR_SHAPE;
    }
    if (sh->T >= (int64_t(1) << 31) || sh->B * sh->T * sh->H >= (int64_t(1) << 31)) return KDA_ERR_SHAPE;
    if (sh->groups < 0 || (sh->groups > 1 && sh->H % sh->groups != 0)) return KDA_ERR_SHAPE;
    return KDA_OK;
}

struct LinLayout {
    size_t share_q, share_k, total;
};
LinLayout layout_of(const kda_linattn_shape* sh, bool backward) {
    LinLayout l;
    size_t o = 1024;   // the status word
    const size_t share = backward && groups_of(sh) > 1 ? align_up((size_t)(sh->B * sh->T * sh->H) * D * sizeof(float), 1024) : 0;
    l.share_q = o; o += share;
    l.share_k = o; o += share;
    l.total = o;
    return l;
}

kda_status common_checks(const kda_linattn_shape* sh, const int64_t* cu, const void* ws, size_t bytes, bool backward) {
    const kda_status st = check_shape(sh, cu != nullptr);
    if (st != KDA_OK) return st;
    if (!ws || bytes < layout_of(sh, backward).total) return KDA_ERR_WORKSPACE;
    if (misaligned(ws) || (reinterpret_cast<uintptr_t>(cu) & 7u)) return KDA_ERR_ALIGN;
    return KDA_OK;
}

void run_jobs(const kda_linattn_shape* sh, LinArgs& a, int jobs, const int64_t* cu, const float* log_decay, uint8_t* ws,
              cudaStream_t s) {
    a.cu = cu;
    a.log_decay = log_decay;
    a.T = sh->T;
    a.H = (int)sh->H;
    a.N = (int)sh->N;
    a.ws = ws;
    linattn_offsets_kernel<<<1, 1024, 0, s>>>(cu, sh->N, sh->B * sh->T, ws);
    linattn_kernel<<<dim3((unsigned)sh->H, (unsigned)sh->N, (unsigned)jobs), 128, 0, s>>>(a);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" size_t kda_linattn_workspace_size(const kda_linattn_shape* shape, int backward) {
    // the same shape may be used with or without offsets
    if (!shape || (check_shape(shape, true) != KDA_OK && check_shape(shape, false) != KDA_OK)) return 0;
    return layout_of(shape, backward != 0).total;
}

extern "C" kda_status kda_linattn_fwd(const kda_linattn_shape* shape, const kda_bf16* q, const kda_bf16* k,
                                      const kda_bf16* v, const float* log_decay, const float* h0,
                                      const int64_t* cu_seqlens, kda_bf16* o, float* hT, void* workspace,
                                      size_t workspace_bytes, void* stream) {
    const kda_status st = common_checks(shape, cu_seqlens, workspace, workspace_bytes, false);
    if (st != KDA_OK) return st;
    if ((shape->B * shape->T > 0 && (!q || !k || !v || !o)) || !log_decay) return KDA_ERR_NULL;
    const void* ptrs[] = {q, k, v, log_decay, h0, o, hT};
    for (const void* p : ptrs)
        if (misaligned(p)) return KDA_ERR_ALIGN;
    const int G = groups_of(shape);
    LinArgs a{};
    a.job[0] = LinJob{q, k, v, G, G, 1, o, nullptr, h0, hT, 0, 0, 1.0f, shape->scale};
    run_jobs(shape, a, 1, cu_seqlens, log_decay, static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream));
    return launched("kda_linattn_fwd launch");
}

extern "C" kda_status kda_linattn_bwd(const kda_linattn_shape* shape, const kda_bf16* q, const kda_bf16* k,
                                      const kda_bf16* v, const float* log_decay, const float* h0,
                                      const int64_t* cu_seqlens, const kda_bf16* do_, const float* dhT, kda_bf16* dq,
                                      kda_bf16* dk, kda_bf16* dv, float* dh0, void* workspace, size_t workspace_bytes,
                                      void* stream) {
    const kda_status st = common_checks(shape, cu_seqlens, workspace, workspace_bytes, true);
    if (st != KDA_OK) return st;
    const int64_t tokens = shape->B * shape->T;
    if ((tokens > 0 && (!q || !k || !v || !do_ || !dq || !dk || !dv)) || !log_decay) return KDA_ERR_NULL;
    const void* ptrs[] = {q, k, v, log_decay, h0, do_, dhT, dq, dk, dv, dh0};
    for (const void* p : ptrs)
        if (misaligned(p)) return KDA_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const int G = groups_of(shape);
    const LinLayout lay = layout_of(shape, true);
    float* const share_q = G > 1 ? reinterpret_cast<float*>(ws + lay.share_q) : nullptr;
    float* const share_k = G > 1 ? reinterpret_cast<float*>(ws + lay.share_k) : nullptr;
    const float sc = shape->scale;
    LinArgs a{};
    a.job[0] = LinJob{do_, v, k, 1, 1, G, dq, share_q, h0, nullptr, 1, 0, 1.0f, sc};
    a.job[1] = LinJob{v, do_, q, 1, 1, G, dk, share_k, dhT, nullptr, 1, 1, sc, 1.0f};
    a.job[2] = LinJob{k, q, do_, G, G, 1, dv, nullptr, dhT, dh0, 0, 1, sc, 1.0f};
    run_jobs(shape, a, 3, cu_seqlens, log_decay, ws, s);
    if (G > 1 && tokens > 0) {
        const int64_t n4 = tokens * (shape->H / G) * (D / 4);
        linattn_group_sum_kernel<<<dim3((unsigned)((n4 + 255) / 256), 2), 256, 0, s>>>(share_q, share_k, dq, dk, n4, G);
    }
    return launched("kda_linattn_bwd launch");
}

extern "C" kda_status kda_linattn_decode(long long n_req, long long H, long long groups, float scale, const kda_bf16* q,
                                         const kda_bf16* k, const kda_bf16* v, const float* log_decay, float* state,
                                         kda_bf16* o, void* stream) {
    if (n_req < 0 || H <= 0 || H > (1 << 20) || n_req > (1LL << 31) - 1 || n_req * H > (1LL << 31) - 1) return KDA_ERR_SHAPE;
    if (groups < 0 || (groups > 1 && H % groups != 0)) return KDA_ERR_SHAPE;
    if (!(std::isfinite(scale) && scale > 0.0f)) return KDA_ERR_UNSUPPORTED;
    if (n_req == 0) return KDA_OK;
    if (!q || !k || !v || !log_decay || !state || !o) return KDA_ERR_NULL;
    const void* ptrs[] = {q, k, v, log_decay, state, o};
    for (const void* p : ptrs)
        if (misaligned(p)) return KDA_ERR_ALIGN;
    const int G = groups > 1 ? (int)groups : 1;
    linattn_decode_kernel<<<(unsigned)(n_req * H), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        q, k, v, log_decay, state, o, (int)H, G, scale);
    return launched("kda_linattn_decode launch");
}
