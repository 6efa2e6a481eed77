// Layer norm over rows, forward and backward, statistics and sums in fp32.
//   y  = (x - mean) rstd w + b
//   dx = rstd (a - mean(a) - xh mean(a xh)),  a = dy w,  xh = (x - mean) rstd
//   dw = sum_rows dy xh,  db = sum_rows dy
// A few operations per byte: HBM bounds all of it, so every input is read once and kept in
// registers between the row's sums and its outputs, and dw, db are summed on the same pass, each
// thread over the rows it meets for columns of its own, in registers. Three forms, by width:
//  - narrow (up to 64 units a row): rows by warps, several at a time, sums by shuffles;
//  - wide (up to 16384 columns): persistent blocks, a row at a time, rows arriving in shared memory
//    by bulk copies some rows ahead;
//  - beyond: a block for each row that reads it again for every step.
// A unit is 16 bytes where the width is a multiple of it, a single element otherwise (bulk copies
// then bring the aligned span around the row, and elements are read one by one from shared memory).
#include <cmath>
#include <cstdio>
#include "kda_internal.cuh"
#include "umma.cuh"

namespace kda {
void set_last_error_text(const char* msg);

namespace {
constexpr int kThreads = 256;
constexpr int kSMs = 152;
constexpr int kWideMost = 16384;       // columns of the wide form
constexpr int kNarrowUnits = 64;       // units of the narrow form with 16-byte units
constexpr int kNarrowColumns = 512;    // and with single elements

__device__ __forceinline__ float get(const uint16_t* p) { return bf2f(*p); }
__device__ __forceinline__ float get(const float* p) { return *p; }
__device__ __forceinline__ void put(uint16_t* p, float x) { *p = f2bf(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }

// A unit in registers as it is stored, and as fp32.
template <typename T, int V> struct Unit;
template <> struct Unit<uint16_t, 8> {
    uint4 r;
    __device__ __forceinline__ void load(const uint16_t* p) { r = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void load_stream(const uint16_t* p) { r = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void zero() { r = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ float at(int i) const {
        const uint32_t w = i < 2 ? r.x : i < 4 ? r.y : i < 6 ? r.z : r.w;
        return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
    }
    __device__ static __forceinline__ void store(uint16_t* p, const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
    }
};
template <> struct Unit<float, 4> {
    float4 r;
    __device__ __forceinline__ void load(const float* p) { r = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void load_stream(const float* p) { r = __ldcs(reinterpret_cast<const float4*>(p)); }
    __device__ __forceinline__ void zero() { r = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    __device__ __forceinline__ float at(int i) const { return i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w; }
    __device__ static __forceinline__ void store(float* p, const float (&f)[4]) {
        __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
    }
};
template <typename T> struct Unit<T, 1> {
    float r;
    __device__ __forceinline__ void load(const T* p) { r = get(p); }
    __device__ __forceinline__ void load_stream(const T* p) { r = get(p); }
    __device__ __forceinline__ void zero() { r = 0.0f; }
    __device__ __forceinline__ float at(int) const { return r; }
    __device__ static __forceinline__ void store(T* p, const float (&f)[1]) { put(p, f[0]); }
};
// the parameters of a unit's columns, `other` without one
template <int V>
__device__ __forceinline__ void params(const float* p, int c, float other, float (&f)[V]) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = other;
    } else if constexpr (V == 1) {
        f[0] = __ldg(p + c);
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(p + c + i));
            f[i] = x.x; f[i + 1] = x.y; f[i + 2] = x.z; f[i + 3] = x.w;
        }
    }
}

// A thread's columns are its own for all rows, so their parameters stay in registers, up to 24 columns
// (they are as long as two or four bf16 rows: fetched for every row, 96 KB of them at a width of 12288
// came from L2 each time and held the forward at 3.1 of 6.7 TB/s).
template <int NV, int V> struct Params {
    static constexpr bool kept = NV * V <= 24;
    const float* p;
    float other;
    float f[kept ? NV : 1][V];
    __device__ __forceinline__ void init(const float* from, float without, int first, int step, int units) {
        p = from;
        other = without;
        if constexpr (kept)
#pragma unroll
            for (int k = 0; k < NV; ++k) params<V>(first + step * k < units ? p : nullptr, (first + step * k) * V, other, f[k]);
    }
    __device__ __forceinline__ void at(int k, int i, float (&o)[V]) const {   // unit k of the thread, unit i of the row
        if constexpr (kept)
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = f[k][e];
        else params<V>(p, i * V, other, o);
    }
};

// ---------------------------------------------------------------------------------- narrow
// Lanes lpr * s .. lpr * (s + 1) - 1 of a warp hold row s of its 32 / lpr rows, lane l of them units
// l, l + 32, .. (lpr < 32: one unit).
__device__ __forceinline__ float lanes_sum(float x, int lpr) {
    for (int o = lpr >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <typename T, int V, int NV>
__global__ void __launch_bounds__(kThreads)
    norm_fwd_narrow_kernel(const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ b, T* __restrict__ y,
                           float* __restrict__ mean, float* __restrict__ rstd, int64_t rows, int width, int units, int lpr,
                           float eps) {
    const int lane = threadIdx.x & 31, sub = lane / lpr, l = lane % lpr, rpw = 32 / lpr;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32), first = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const float inv = 1.0f / (float)width;
    Params<NV, V> pw, pb;
    pw.init(w, 1.0f, l, 32, units);
    pb.init(b, 0.0f, l, 32, units);
    for (int64_t r0 = first * rpw; r0 < rows; r0 += warps * rpw) {
        const int64_t r = r0 + sub;
        const bool in = r < rows;
        Unit<T, V> u[NV];
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = l + 32 * k;
            if (in && i < units) u[k].load_stream(x + r * width + i * V);
            else u[k].zero();
#pragma unroll
            for (int e = 0; e < V; ++e) s += u[k].at(e);
        }
        const float mu = lanes_sum(s, lpr) * inv;
        s = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (l + 32 * k < units)
#pragma unroll
                for (int e = 0; e < V; ++e) s += (u[k].at(e) - mu) * (u[k].at(e) - mu);
        const float rs = rsqrtf(lanes_sum(s, lpr) * inv + eps);
        if (!in) continue;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = l + 32 * k;
            if (i < units) {
                float wv[V], bv[V], o[V];
                pw.at(k, i, wv);
                pb.at(k, i, bv);
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] = (u[k].at(e) - mu) * rs * wv[e] + bv[e];
                Unit<T, V>::store(y + r * width + i * V, o);
            }
        }
        if (l == 0) {
            if (mean) mean[r] = mu;
            if (rstd) rstd[r] = rs;
        }
    }
}

template <typename T, int V, int NV, int R>   // R: row groups in flight
__global__ void __launch_bounds__(kThreads, V * NV <= 8 ? 4 : 2)
    norm_bwd_narrow_kernel(const T* __restrict__ x, const T* __restrict__ dy, const float* __restrict__ w,
                           const float* __restrict__ mean, const float* __restrict__ rstd, T* __restrict__ dx,
                           float* __restrict__ part, int64_t rows, int width, int units, int lpr) {
    extern __shared__ float acc[];   // [warps][2][width]
    grid_launch_next();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / lpr, l = lane % lpr, rpw = 32 / lpr;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32), first = (int64_t)blockIdx.x * (kThreads / 32) + warp;
    const float inv = 1.0f / (float)width;
    float wv[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        params<V>(w, l + 32 * k < units ? (l + 32 * k) * V : 0, 1.0f, wv[k]);
#pragma unroll
        for (int e = 0; e < V; ++e) dw[k][e] = db[k][e] = 0.0f;
    }
    for (int64_t r0 = first * rpw; r0 < rows; r0 += R * warps * rpw) {
        Unit<T, V> ux[R][NV], ug[R][NV];
        float mu[R], rs[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int64_t r = r0 + q * warps * rpw + sub;
            const bool in = r < rows;
            mu[q] = in ? mean[r] : 0.0f;
            rs[q] = in ? rstd[r] : 0.0f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int i = l + 32 * k;
                if (in && i < units) {
                    ux[q][k].load_stream(x + r * width + i * V);
                    ug[q][k].load_stream(dy + r * width + i * V);
                } else {
                    ux[q][k].zero();
                    ug[q][k].zero();
                }
            }
        }
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int64_t r = r0 + q * warps * rpw + sub;
            float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float g = ug[q][k].at(e), h = (ux[q][k].at(e) - mu[q]) * rs[q], a = g * wv[k][e];
                    s1 += a;
                    s2 += a * h;
                    dw[k][e] += g * h;
                    db[k][e] += g;
                }
            s1 = lanes_sum(s1, lpr) * inv;
            s2 = lanes_sum(s2, lpr) * inv;
            if (r < rows)
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int i = l + 32 * k;
                    if (i < units) {
                        float o[V];
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            o[e] = rs[q] * (ug[q][k].at(e) * wv[k][e] - s1 - (ux[q][k].at(e) - mu[q]) * rs[q] * s2);
                        Unit<T, V>::store(dx + r * width + i * V, o);
                    }
                }
        }
    }
    if (!part) return;
    // the warp's rows by lane, then the block's warps in order
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e)
            for (int o = lpr; o < 32; o <<= 1) {
                dw[k][e] += __shfl_xor_sync(0xffffffffu, dw[k][e], o);
                db[k][e] += __shfl_xor_sync(0xffffffffu, db[k][e], o);
            }
    if (sub == 0)
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (l + 32 * k < units)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    acc[(size_t)(2 * warp) * width + (l + 32 * k) * V + e] = dw[k][e];
                    acc[(size_t)(2 * warp + 1) * width + (l + 32 * k) * V + e] = db[k][e];
                }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * width; c += kThreads) {
        float s = 0.0f;
        for (int i = 0; i < kThreads / 32; ++i) s += acc[(size_t)2 * i * width + c];
        part[(size_t)blockIdx.x * 2 * width + c] = s;
    }
}

// ------------------------------------------------------------------------------------ wide
__device__ __forceinline__ float2 warp_sums(float a, float b) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    return make_float2(a, b);
}
// the sum of the block's warps' pairs, four at a time; what lies past them in the 32 does not count
__device__ __forceinline__ float2 sum_of(const float2 (&buf)[32]) {
    float2 s = make_float2(0.0f, 0.0f);
    const int n = blockDim.x >> 5;
    for (int i = 0; i < n; i += 4) {
        const float4 p = *reinterpret_cast<const float4*>(&buf[i]), q = *reinterpret_cast<const float4*>(&buf[i + 2]);
        s.x += (p.x + (i + 1 < n ? p.z : 0.0f)) + ((i + 2 < n ? q.x : 0.0f) + (i + 3 < n ? q.z : 0.0f));
        s.y += (p.y + (i + 1 < n ? p.w : 0.0f)) + ((i + 2 < n ? q.y : 0.0f) + (i + 3 < n ? q.w : 0.0f));
    }
    return s;
}
// sums over the block, the same values in every thread, with one barrier (the caller uses two buffers in turn)
__device__ __forceinline__ float2 block_sums(float a, float b, float2 (&buf)[32]) {
    const float2 p = warp_sums(a, b);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = p;
    __syncthreads();
    return sum_of(buf);
}
// rows at a time of the backward, by a thread's columns (single elements take a register each)
__host__ __device__ constexpr int bwd_rows(int columns, bool vec) { return columns <= (vec ? 16 : 8) ? 2 : 1; }

// Rows on their way to shared memory: a step of R rows (r, r + stride, ..) of each input, `stages` steps
// ahead, of each row the aligned span around it. The last bytes of a tensor whose size is no multiple of
// 16 are not copied: take() reads them from global memory.
template <int R>
struct Rows {
    uint8_t* at;             // [stages][inputs][R][pitch]
    uint64_t* full;          // [stages]
    size_t row_bytes, most;  // most: the tensor's size rounded down to 16 bytes
    int64_t rows, stride;
    int pitch, inputs;
    __device__ __forceinline__ void issue(int64_t r0, int stage, const void* a, const void* b) const {
        uint32_t n[R], sum = 0;
        size_t from[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int64_t r = r0 + q * stride;
            const size_t p = (size_t)r * row_bytes;
            size_t to = (p + row_bytes + 15) & ~(size_t)15;
            from[q] = p & ~(size_t)15;
            if (to > most) to = most;
            n[q] = r < rows && to > from[q] ? (uint32_t)(to - from[q]) : 0u;
            sum += n[q];
        }
        mbar_arrive_expect_tx(&full[stage], sum * (uint32_t)inputs);
#pragma unroll
        for (int q = 0; q < R; ++q)
            if (n[q]) {
                bulk_g2s(slot(stage, 0, q), static_cast<const uint8_t*>(a) + from[q], n[q], &full[stage]);
                if (inputs > 1) bulk_g2s(slot(stage, 1, q), static_cast<const uint8_t*>(b) + from[q], n[q], &full[stage]);
            }
    }
    __device__ __forceinline__ uint8_t* slot(int stage, int input, int q) const {
        return at + ((size_t)(stage * inputs + input) * R + q) * pitch;
    }
    // element 0 of row r, the q-th of its step, of an input in shared memory
    template <typename T>
    __device__ __forceinline__ const T* row(int64_t r, int stage, int input, int q) const {
        return reinterpret_cast<const T*>(slot(stage, input, q) + (((size_t)r * row_bytes) & 15));
    }
};
// a unit of the row from shared memory, or from global memory past the copied part
template <typename T, int V, int R>
__device__ __forceinline__ void take(Unit<T, V>& u, const Rows<R>& m, const T* in_smem, const T* in_global, int64_t r, int c) {
    if (V == 1 && (size_t)r * m.row_bytes + (size_t)(c + 1) * sizeof(T) > m.most) u.load(in_global + c);
    else u.load(in_smem + c);
}
template <int R>
__device__ __forceinline__ Rows<R> rows_of(uint8_t* smem, size_t row_bytes, int64_t rows, int pitch, int inputs) {
    Rows<R> m;
    m.full = reinterpret_cast<uint64_t*>(smem);
    m.at = smem + 64;
    m.row_bytes = row_bytes;
    m.most = (row_bytes * (size_t)rows) & ~(size_t)15;
    m.rows = rows;
    m.stride = gridDim.x;
    m.pitch = pitch;
    m.inputs = inputs;
    return m;
}

// Persistent blocks: rows blockIdx.x, + gridDim.x, .., two at a time (their sums share the barriers, and one's
// arithmetic runs in the other's waits: one row at a time took 81 instead of .. us at 8192 x 12288); thread t
// holds units t, t + blockDim.x, .. A copy that has not arrived after 2 s leaves NaN in its rows' outputs
// (there is no workspace to report it in).
template <typename T, int V, int NV>
__global__ void __launch_bounds__(512)
    norm_fwd_wide_kernel(const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ b, T* __restrict__ y,
                         float* __restrict__ mean, float* __restrict__ rstd, int64_t rows, int width, int units, int pitch,
                         int stages, float eps) {
    constexpr int R = 2;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float2 buf[2][32];
    const Rows<R> m = rows_of<R>(smem, (size_t)width * sizeof(T), rows, pitch, 1);
    const int t = threadIdx.x, nt = blockDim.x;
    const int64_t step = (int64_t)R * gridDim.x;
    const float inv = 1.0f / (float)width;
    if (t == 0) {
        for (int i = 0; i < stages; ++i) mbar_init(&m.full[i], 1);
        fence_mbar_init();
        for (int i = 0; i < stages; ++i)
            if (blockIdx.x + i * step < rows) m.issue(blockIdx.x + i * step, i, x, nullptr);
    }
    Params<NV, V> pw, pb;
    pw.init(w, 1.0f, t, nt, units);
    pb.init(b, 0.0f, t, nt, units);
    __syncthreads();
    int stage = 0;
    uint32_t phase = 0;
    for (int64_t r = blockIdx.x; r < rows; r += step) {
        const bool ok = mbar_wait(&m.full[stage], phase);
        Unit<T, V> u[R][NV];
        float s[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int64_t rq = r + q * m.stride;
            const T* row = m.template row<T>(rq, stage, 0, q);
            s[q] = 0.0f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int i = t + nt * k;
                if (i < units && rq < rows) take(u[q][k], m, row, x + rq * width, rq, i * V);
                else u[q][k].zero();
#pragma unroll
                for (int e = 0; e < V; ++e) s[q] += u[q][k].at(e);
            }
        }
        const float2 mu2 = block_sums(ok ? s[0] : __int_as_float(0x7fffffff), ok ? s[1] : __int_as_float(0x7fffffff), buf[0]);
        const float mu[R] = {mu2.x * inv, mu2.y * inv};
        // every thread has its part of the rows in registers: the stage takes later ones
        const int64_t next = r + stages * step;
        if (t == 0 && next < rows) m.issue(next, stage, x, nullptr);
#pragma unroll
        for (int q = 0; q < R; ++q) {
            s[q] = 0.0f;
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (t + nt * k < units)
#pragma unroll
                    for (int e = 0; e < V; ++e) s[q] += (u[q][k].at(e) - mu[q]) * (u[q][k].at(e) - mu[q]);
        }
        const float2 var = block_sums(s[0], s[1], buf[1]);
        const float rs[R] = {rsqrtf(var.x * inv + eps), rsqrtf(var.y * inv + eps)};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = t + nt * k;
            if (i < units) {
                float wv[V], bv[V], o[V];
                pw.at(k, i, wv);
                pb.at(k, i, bv);
#pragma unroll
                for (int q = 0; q < R; ++q) {
                    const int64_t rq = r + q * m.stride;
#pragma unroll
                    for (int e = 0; e < V; ++e) o[e] = (u[q][k].at(e) - mu[q]) * rs[q] * wv[e] + bv[e];
                    if (rq < rows) Unit<T, V>::store(y + rq * width + i * V, o);
                }
            }
        }
        if (t < R && r + t * m.stride < rows) {
            if (mean) mean[r + t * m.stride] = t == 0 ? mu[0] : mu[1];
            if (rstd) rstd[r + t * m.stride] = t == 0 ? rs[0] : rs[1];
        }
        if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
        }
    }
}

// The same for the backward, with dw and db of a thread's columns in registers; two rows at a time where
// registers allow.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(512)
    norm_bwd_wide_kernel(const T* __restrict__ x, const T* __restrict__ dy, const float* __restrict__ w,
                         const float* __restrict__ mean, const float* __restrict__ rstd, T* __restrict__ dx,
                         float* __restrict__ part, int64_t rows, int width, int units, int pitch, int stages) {
    constexpr int R = bwd_rows(NV * V, V > 1);
    grid_launch_next();
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float2 buf[2][R][32];
    const Rows<R> m = rows_of<R>(smem, (size_t)width * sizeof(T), rows, pitch, 2);
    const int t = threadIdx.x, nt = blockDim.x;
    const int64_t step = (int64_t)R * gridDim.x;
    const float inv = 1.0f / (float)width;
    if (t == 0) {
        for (int i = 0; i < stages; ++i) mbar_init(&m.full[i], 1);
        fence_mbar_init();
        for (int i = 0; i < stages; ++i)
            if (blockIdx.x + i * step < rows) m.issue(blockIdx.x + i * step, i, x, dy);
    }
    float dw[NV][V], db[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) dw[k][e] = db[k][e] = 0.0f;
    Params<NV, V> pw;
    pw.init(w, 1.0f, t, nt, units);
    __syncthreads();
    int stage = 0, turn = 0;
    uint32_t phase = 0;
    float mu_next[R], rs_next[R];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int64_t rq = r + q * m.stride;
            mu_next[q] = rq < rows ? mean[rq] : 0.0f;
            rs_next[q] = rq < rows ? rstd[rq] : 0.0f;
        }
    };
    fetch(blockIdx.x);
    for (int64_t r = blockIdx.x; r < rows; r += step) {
        float mu[R], rs[R], s1[R], s2[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            mu[q] = mu_next[q];
            rs[q] = rs_next[q];
            s1[q] = s2[q] = 0.0f;
        }
        fetch(r + step);
        const bool ok = mbar_wait(&m.full[stage], phase);
        Unit<T, V> ux[R][NV], ug[R][NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = t + nt * k;
            float wv[V];
            if (i < units) pw.at(k, i, wv);
#pragma unroll
            for (int q = 0; q < R; ++q) {
                const int64_t rq = r + q * m.stride;
                if (i < units && rq < rows) {
                    take(ux[q][k], m, m.template row<T>(rq, stage, 0, q), x + rq * width, rq, i * V);
                    take(ug[q][k], m, m.template row<T>(rq, stage, 1, q), dy + rq * width, rq, i * V);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float g = ug[q][k].at(e), h = (ux[q][k].at(e) - mu[q]) * rs[q], a = g * wv[e];
                        s1[q] += a;
                        s2[q] += a * h;
                        dw[k][e] += g * h;
                        db[k][e] += g;
                    }
                }
            }
        }
        // one barrier for the sums of all rows of the step
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const float2 p = warp_sums(ok ? s1[q] : __int_as_float(0x7fffffff), s2[q]);
            if ((t & 31) == 0) buf[turn][q][t >> 5] = p;
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const float2 p = sum_of(buf[turn][q]);
            s1[q] = p.x * inv;
            s2[q] = p.y * inv;
        }
        turn ^= 1;
        const int64_t next = r + stages * step;
        if (t == 0 && next < rows) m.issue(next, stage, x, dy);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = t + nt * k;
            if (i < units) {
                float wv[V], o[V];
                pw.at(k, i, wv);
#pragma unroll
                for (int q = 0; q < R; ++q) {
                    const int64_t rq = r + q * m.stride;
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        o[e] = rs[q] * (ug[q][k].at(e) * wv[e] - s1[q] - (ux[q][k].at(e) - mu[q]) * rs[q] * s2[q]);
                    if (rq < rows) Unit<T, V>::store(dx + rq * width + i * V, o);
                }
            }
        }
        if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
        }
    }
    if (!part) return;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int i = t + nt * k;
        if (i < units)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                part[(size_t)blockIdx.x * 2 * width + i * V + e] = dw[k][e];
                part[((size_t)blockIdx.x * 2 + 1) * width + i * V + e] = db[k][e];
            }
    }
}

// ---------------------------------------------------------------------------- any width
// One row for each block, read three times (from the cache after the first).
__device__ __forceinline__ float block_sum(float x, float2 (&buf)[32]) {
    const float s = block_sums(x, 0.0f, buf).x;
    __syncthreads();
    return s;
}
template <typename T>
__global__ void __launch_bounds__(kThreads)
    norm_fwd_any_kernel(const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ b, T* __restrict__ y,
                        float* __restrict__ mean, float* __restrict__ rstd, int64_t rows, int width, float eps) {
    __shared__ __align__(16) float2 buf[32];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T* xr = x + r * width;
        float s = 0.0f;
        for (int c = threadIdx.x; c < width; c += kThreads) s += get(xr + c);
        const float mu = block_sum(s, buf) / (float)width;
        s = 0.0f;
        for (int c = threadIdx.x; c < width; c += kThreads) {
            const float d = get(xr + c) - mu;
            s += d * d;
        }
        const float rs = rsqrtf(block_sum(s, buf) / (float)width + eps);
        for (int c = threadIdx.x; c < width; c += kThreads)
            put(y + r * width + c, (get(xr + c) - mu) * rs * (w ? w[c] : 1.0f) + (b ? b[c] : 0.0f));
        if (threadIdx.x == 0) {
            if (mean) mean[r] = mu;
            if (rstd) rstd[r] = rs;
        }
    }
}
template <typename T>
__global__ void __launch_bounds__(kThreads)
    norm_dx_any_kernel(const T* __restrict__ x, const T* __restrict__ dy, const float* __restrict__ w,
                       const float* __restrict__ mean, const float* __restrict__ rstd, T* __restrict__ dx, int64_t rows,
                       int width) {
    __shared__ __align__(16) float2 buf[2][32];
    int turn = 0;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x, turn ^= 1) {
        const float mu = mean[r], rs = rstd[r];
        float s1 = 0.0f, s2 = 0.0f;
        for (int c = threadIdx.x; c < width; c += kThreads) {
            const float a = get(dy + r * width + c) * (w ? w[c] : 1.0f);
            s1 += a;
            s2 += a * ((get(x + r * width + c) - mu) * rs);
        }
        const float2 s = block_sums(s1, s2, buf[turn]);
        s1 = s.x / (float)width;
        s2 = s.y / (float)width;
        for (int c = threadIdx.x; c < width; c += kThreads) {
            const float a = get(dy + r * width + c) * (w ? w[c] : 1.0f);
            put(dx + r * width + c, rs * (a - s1 - (get(x + r * width + c) - mu) * rs * s2));
        }
    }
}
// block (i, j): 256 columns, every gridDim.y-th row
template <typename T>
__global__ void __launch_bounds__(kThreads)
    norm_dw_any_kernel(const T* __restrict__ x, const T* __restrict__ dy, const float* __restrict__ mean,
                       const float* __restrict__ rstd, float* __restrict__ part, int64_t rows, int width) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= width) return;
    float dw = 0.0f, db = 0.0f;
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
        const float g = get(dy + r * width + c);
        dw += g * ((get(x + r * width + c) - mean[r]) * rstd[r]);
        db += g;
    }
    part[((size_t)blockIdx.y * 2) * width + c] = dw;
    part[((size_t)blockIdx.y * 2 + 1) * width + c] = db;
}

// dw and db from the n blocks' sums: 32 columns a block, 32 row groups that each add every 32nd partial,
// then the groups in order.
__global__ void __launch_bounds__(1024)
    norm_reduce_kernel(const float* __restrict__ part, int n, int width, float* __restrict__ dw, float* __restrict__ db) {
    grid_wait_before();
    __shared__ float s[32][33];
    float* const out = blockIdx.y ? db : dw;
    if (!out) return;
    const int c = blockIdx.x * 32 + threadIdx.x;
    float a = 0.0f;
    if (c < width)
#pragma unroll 8
        for (int i = threadIdx.y; i < n; i += 32) a += part[((size_t)i * 2 + blockIdx.y) * width + c];
    s[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    if (threadIdx.y == 0 && c < width) {
        a = 0.0f;
        for (int i = 0; i < 32; ++i) a += s[i][threadIdx.x];
        out[c] = a;
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

bool valid_size(long long rows, long long width) {
    return rows >= 0 && width >= 1 && width <= (1LL << 20) && rows <= (1LL << 40) / width;
}

// Most blocks whose sums of dw and db are kept: four on an SM, and one for every SM at least. Their sums are
// written and read again, so they stay below about a twentieth of what the rows themselves move.
constexpr int kMostParts = 4 * kSMs;
int most_parts(long long rows, size_t size) {
    const long long n = rows * (long long)size / 54;
    return (int)(n < kSMs ? kSMs : n > kMostParts ? kMostParts : n);
}

// Which form a width takes, and its launch.
struct Form {
    int units, lpr, nv;      // lpr: lanes of a row (narrow), 0: wide or any
    bool vec, wide;
    int threads, pitch, stages, per_sm;
    size_t smem;
};
Form form_of(long long width, size_t size, int inputs) {
    Form f{};
    const int v = (int)(16 / size);
    f.vec = width % v == 0;
    f.units = (int)(f.vec ? width / v : width);
    if (f.vec ? f.units <= kNarrowUnits : width <= kNarrowColumns) {
        f.lpr = 1;
        while (f.lpr < f.units && f.lpr < 32) f.lpr *= 2;
        const int need = (f.units + 31) / 32;
        f.nv = 1;
        while (f.nv < need) f.nv *= 2;
        return f;
    }
    if (width > kWideMost) return f;
    f.wide = true;
    // 16 bf16 or 8 fp32 columns a thread and small blocks, so that many rows are in flight; more columns
    // where 512 threads do not hold the row
    const int most[] = {2, 3, 4, 8, 16, 32};
    for (int nv : most) {
        f.nv = nv;
        if ((f.vec || nv >= 8) && f.units <= nv * 512) break;
    }
    f.threads = ((f.units + f.nv - 1) / f.nv + 31) / 32 * 32;
    f.pitch = (int)((width * size + 31) / 16 * 16);
    const int columns = f.nv * (f.vec ? v : 1);
    const int stage = f.pitch * inputs * (inputs == 1 ? 2 : bwd_rows(columns, f.vec));
    const int room = columns * (inputs + 1) >= 48 ? 512 : 1024;   // threads on an SM, by registers
    f.per_sm = room / f.threads < 1 ? 1 : room / f.threads;
    if (f.per_sm > 16) f.per_sm = 16;
    // up to four steps ahead, within the SM's shared memory; fewer blocks rather than none ahead
    for (;; --f.per_sm) {
        f.stages = (int)(((size_t)216 * 1024 / f.per_sm - 1024 - 64) / stage);
        if (f.stages >= 2 || f.per_sm == 1) break;
    }
    if (f.stages > 4) f.stages = 4;
    if (f.stages < 1) f.stages = 1;
    f.smem = 64 + (size_t)stage * f.stages;
    return f;
}

unsigned blocks(long long rows, long long most) { return (unsigned)(rows < most ? rows : most); }

template <typename T, int V, int NV>
kda_status fwd_wide(const Form& f, long long rows, int width, float eps, const T* x, const float* w, const float* b, T* y,
                    float* mean, float* rstd, cudaStream_t s) {
    auto k = norm_fwd_wide_kernel<T, V, NV>;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)f.smem) != cudaSuccess) return launched("kda_layernorm_fwd");
    k<<<blocks(rows, (long long)kSMs * f.per_sm), f.threads, f.smem, s>>>(x, w, b, y, mean, rstd, rows, width, f.units, f.pitch,
                                                                       f.stages, eps);
    return launched("kda_layernorm_fwd launch");
}
template <typename T, int V, int NV>
kda_status fwd_narrow(const Form& f, long long rows, int width, float eps, const T* x, const float* w, const float* b, T* y,
                      float* mean, float* rstd, cudaStream_t s) {
    const long long rpb = (long long)(kThreads / 32) * (32 / f.lpr);
    norm_fwd_narrow_kernel<T, V, NV><<<blocks((rows + rpb - 1) / rpb, 8LL * kSMs), kThreads, 0, s>>>(x, w, b, y, mean, rstd, rows,
                                                                                                     width, f.units, f.lpr, eps);
    return launched("kda_layernorm_fwd launch");
}
template <typename T>
kda_status fwd(long long rows, int width, float eps, const void* xv, const float* w, const float* b, void* yv, float* mean,
               float* rstd, cudaStream_t s) {
    const T* x = static_cast<const T*>(xv);
    T* y = static_cast<T*>(yv);
    constexpr int V = 16 / sizeof(T);
    const Form f = form_of(width, sizeof(T), 1);
#define KDA_NORM(fn, v, n) return fn<T, v, n>(f, rows, width, eps, x, w, b, y, mean, rstd, s)
    if (f.lpr && f.vec) {
        if (f.nv == 1) KDA_NORM(fwd_narrow, V, 1);
        KDA_NORM(fwd_narrow, V, 2);
    }
    if (f.lpr) {
        if (f.nv <= 2) KDA_NORM(fwd_narrow, 1, 2);
        if (f.nv <= 4) KDA_NORM(fwd_narrow, 1, 4);
        if (f.nv <= 8) KDA_NORM(fwd_narrow, 1, 8);
        KDA_NORM(fwd_narrow, 1, 16);
    }
    if (f.wide && f.vec) {
        if (f.nv == 2) KDA_NORM(fwd_wide, V, 2);
        if (f.nv == 3) KDA_NORM(fwd_wide, V, 3);
        if (f.nv == 4) KDA_NORM(fwd_wide, V, 4);
        if constexpr (V == 4) KDA_NORM(fwd_wide, V, 8);
    }
    if (f.wide) {
        if (f.nv <= 8) KDA_NORM(fwd_wide, 1, 8);
        if (f.nv <= 16) KDA_NORM(fwd_wide, 1, 16);
        KDA_NORM(fwd_wide, 1, 32);
    }
#undef KDA_NORM
    norm_fwd_any_kernel<T><<<blocks(rows, 1 << 30), kThreads, 0, s>>>(x, w, b, y, mean, rstd, rows, width, eps);
    return launched("kda_layernorm_fwd launch");
}

template <typename T, int V, int NV>
kda_status bwd_wide(const Form& f, long long rows, int width, const T* x, const T* dy, const float* w, const float* mean,
                    const float* rstd, T* dx, float* part, int* parts, cudaStream_t s) {
    auto k = norm_bwd_wide_kernel<T, V, NV>;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)f.smem) != cudaSuccess) return launched("kda_layernorm_bwd");
    const long long most = (long long)kSMs * f.per_sm, keep = most_parts(rows, sizeof(T));
    *parts = (int)blocks(rows, most < keep ? most : keep);
    k<<<*parts, f.threads, f.smem, s>>>(x, dy, w, mean, rstd, dx, part, rows, width, f.units, f.pitch, f.stages);
    return launched("kda_layernorm_bwd launch");
}
template <typename T, int V, int NV>
kda_status bwd_narrow(const Form& f, long long rows, int width, const T* x, const T* dy, const float* w, const float* mean,
                      const float* rstd, T* dx, float* part, int* parts, cudaStream_t s) {
    constexpr int R = V * NV <= 8 ? 2 : 1;
    const long long rpb = (long long)(kThreads / 32) * (32 / f.lpr);
    *parts = (int)blocks((rows + rpb - 1) / rpb, (V * NV <= 8 ? 4 : 2) * kSMs);   // as many as are resident
    norm_bwd_narrow_kernel<T, V, NV, R><<<*parts, kThreads, (size_t)(kThreads / 32) * 2 * width * sizeof(float), s>>>(
        x, dy, w, mean, rstd, dx, part, rows, width, f.units, f.lpr);
    return launched("kda_layernorm_bwd launch");
}
// dx and, to part where it is given, the sums of `parts` blocks
template <typename T>
kda_status bwd(long long rows, int width, const void* xv, const void* dyv, const float* w, const float* mean, const float* rstd,
               void* dxv, float* part, int* parts, cudaStream_t s) {
    const T *x = static_cast<const T*>(xv), *dy = static_cast<const T*>(dyv);
    T* dx = static_cast<T*>(dxv);
    constexpr int V = 16 / sizeof(T);
    const Form f = form_of(width, sizeof(T), 2);
#define KDA_NORM(fn, v, n) return fn<T, v, n>(f, rows, width, x, dy, w, mean, rstd, dx, part, parts, s)
    if (f.lpr && f.vec) {
        if (f.nv == 1) KDA_NORM(bwd_narrow, V, 1);
        KDA_NORM(bwd_narrow, V, 2);
    }
    if (f.lpr) {
        if (f.nv <= 2) KDA_NORM(bwd_narrow, 1, 2);
        if (f.nv <= 4) KDA_NORM(bwd_narrow, 1, 4);
        if (f.nv <= 8) KDA_NORM(bwd_narrow, 1, 8);
        KDA_NORM(bwd_narrow, 1, 16);
    }
    if (f.wide && f.vec) {
        if (f.nv == 2) KDA_NORM(bwd_wide, V, 2);
        if (f.nv == 3) KDA_NORM(bwd_wide, V, 3);
        if (f.nv == 4) KDA_NORM(bwd_wide, V, 4);
        if constexpr (V == 4) KDA_NORM(bwd_wide, V, 8);
    }
    if (f.wide) {
        if (f.nv <= 8) KDA_NORM(bwd_wide, 1, 8);
        if (f.nv <= 16) KDA_NORM(bwd_wide, 1, 16);
        KDA_NORM(bwd_wide, 1, 32);
    }
#undef KDA_NORM
    norm_dx_any_kernel<T><<<blocks(rows, 1 << 30), kThreads, 0, s>>>(x, dy, w, mean, rstd, dx, rows, width);
    *parts = (int)blocks(rows, kSMs);
    if (part)
        norm_dw_any_kernel<T><<<dim3((unsigned)((width + kThreads - 1) / kThreads), (unsigned)*parts), kThreads, 0, s>>>(
            x, dy, mean, rstd, part, rows, width);
    return launched("kda_layernorm_bwd launch");
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
    return dtype == KDA_BF16 ? fwd<uint16_t>(rows, (int)width, eps, x, weight, bias, y, mean, rstd, s)
                             : fwd<float>(rows, (int)width, eps, x, weight, bias, y, mean, rstd, s);
}

extern "C" size_t kda_layernorm_workspace_size(long long rows, long long width) {
    if (!valid_size(rows, width)) return 0;
    return align_up((size_t)(rows < kMostParts ? rows + 1 : kMostParts) * 2 * (size_t)width * sizeof(float), 1024);
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
    const bool sums = dweight || dbias;
    float* part = sums ? static_cast<float*>(workspace) : nullptr;
    int parts = 0;
    if (rows > 0) {
        const kda_status st = dtype == KDA_BF16
                                  ? bwd<uint16_t>(rows, (int)width, x, dy, weight, mean, rstd, dx, part, &parts, s)
                                  : bwd<float>(rows, (int)width, x, dy, weight, mean, rstd, dx, part, &parts, s);
        if (st != KDA_OK) return st;
    }
    if (sums)
        launch_kernel(norm_reduce_kernel, dim3((unsigned)((width + 31) / 32), 2), dim3(32, 32), 0, s, parts > 0,
                      static_cast<const float*>(workspace), parts, (int)width, dweight, dbias);
    return launched("kda_layernorm_bwd launch");
}
