// Layer norm over rows, forward and backward, statistics and sums in fp32.
//   y  = (x - mean) rstd w + b
//   dx = rstd (a - mean(a) - xh mean(a xh)),  a = dy w,  xh = (x - mean) rstd
//   dw = sum_rows dy xh,  db = sum_rows dy
// A few operations per byte: HBM is the floor of all of it, so every input is read once and kept in
// registers between the row's sums and its outputs, and dw, db are summed on the same pass, each
// thread over the rows it meets for columns of its own, in registers. Three forms, by width:
//  - narrow (up to 64 units a row): rows by warps, several at a time, sums by shuffles;
//  - wide (up to 16384 columns): persistent blocks, one or two rows at a time, rows arriving in shared
//    memory by bulk copies some rows ahead;
//  - beyond: a block for each row that reads it again for every step.
// Measured, of what is read and written once: forward 8192 x 12288 bf16 72 us (5.6 TB/s, of 6.7 that a copy reaches),
// 131072 x 128 bf16 19.7 us (3.4); backward 4099 x 4096 fp32 40 us (5.0), of which 5 are the sum over blocks, 131072 x
// 128 bf16 24 us (4.2), 8192 x 4096 bf16 54 us (3.8), 16384 x 1024 bf16 32 us (3.2); ragged widths take two to four times
// their floor (forward 8192 x 4097 bf16 46 us, 32768 x 501 31; backward 100000 x 131 48). What bounds them is not HBM (14% to
// 62% of its peak in the kernels): the registers that rows are held in leave 16 of 64 warps on an SM, and these issue in
// half of the cycles (45% to 57%) and wait in the others, for the row's sums (barriers, shuffles) and for loads.
// dw and db are sums of a thread's rows in turn, of up to 608 blocks' by 32 groups, of the groups': in fp32 1.5e-7 of their
// size off at 4099 x 4096 (elementary tensor operations: 1.2e-7), 1.6e-7 at 131072 x 128 in bf16 (3.7e-7).
// A unit is 16 aligned bytes. Where the width is no multiple of it, rows start inside a unit, each at one of
// eight (bf16) or four (fp32) places; a thread meets only rows that start at the same place, so that its columns
// stay its own, and its first and last unit of a row hold elements of the neighbours, which do not count.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>
#include "kda_internal.cuh"
#include "umma_bf16.cuh"

namespace kda {
void set_last_error_text(const char* msg);

namespace {
constexpr int kThreads = 256;
constexpr int kSMs = 152;
constexpr int kWideMost = 16384;       // columns of the wide form
constexpr int kNarrowUnits = 64;       // units of the narrow form

__device__ __forceinline__ float get(const uint16_t* p) { return bf2f(*p); }
__device__ __forceinline__ float get(const float* p) { return *p; }
__device__ __forceinline__ void put(uint16_t* p, float x) { *p = f2bf(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }

// A unit, 16 bytes, in registers as it is stored, and as P pairs of fp32 (packed arithmetic: half the instructions).
template <typename T> struct Unit;
template <> struct Unit<uint16_t> {
    static constexpr int V = 8, P = 4;
    uint4 r;
    __device__ __forceinline__ void load(const uint16_t* p) { r = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void load_stream(const uint16_t* p) { r = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void zero() { r = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ f32x2 at(int i) const {   // elements 2 i and 2 i + 1
        const uint32_t w = i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w;
        return two(w << 16, w & 0xffff0000u);
    }
    __device__ __forceinline__ void keep(uint32_t ok) {   // the elements of these bits, zero elsewhere
        r.x &= ((ok & 1u) ? 0xffffu : 0u) | ((ok & 2u) ? 0xffff0000u : 0u);
        r.y &= ((ok & 4u) ? 0xffffu : 0u) | ((ok & 8u) ? 0xffff0000u : 0u);
        r.z &= ((ok & 16u) ? 0xffffu : 0u) | ((ok & 32u) ? 0xffff0000u : 0u);
        r.w &= ((ok & 64u) ? 0xffffu : 0u) | ((ok & 128u) ? 0xffff0000u : 0u);
    }
    __device__ __forceinline__ void load_some(const uint16_t* p, uint32_t ok) {
        uint32_t e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = (ok >> i) & 1u ? p[i] : 0u;
        r = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
    }
    __device__ static __forceinline__ uint32_t pack(f32x2 f) {
        const float2 x = parts(f);
        const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ static __forceinline__ void store(uint16_t* p, const f32x2 (&f)[4]) {
        __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack(f[0]), pack(f[1]), pack(f[2]), pack(f[3])));
    }
    // the first or last elements of a unit (ok) in as few stores as their number has bits, others one by one
    __device__ static __forceinline__ void store_some(uint16_t* p, const f32x2 (&f)[4], uint32_t ok) {
        const uint32_t w[4] = {pack(f[0]), pack(f[1]), pack(f[2]), pack(f[3])};
        if ((ok & 15u) == 15u) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        if ((ok >> 4) == 15u) *reinterpret_cast<uint2*>(p + 4) = make_uint2(w[2], w[3]);
        const bool upper = (ok & 15u) == 0u || (ok & 15u) == 15u;    // the half that is not done
        const uint32_t a = upper ? w[2] : w[0], b = upper ? w[3] : w[1], r = upper ? ok >> 4 : ok & 15u;
        if (!upper && ok >> 4 && ok >> 4 != 15u) {                   // a row inside a unit
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if ((ok >> (4 + i)) & 1u) p[4 + i] = (uint16_t)(i & 1 ? w[2 + i / 2] >> 16 : w[2 + i / 2]);
        }
        if (r == 15u) return;
        uint16_t* const h = p + (upper ? 4 : 0);
        if ((r & 3u) == 3u) *reinterpret_cast<uint32_t*>(h) = a;
        if ((r & 12u) == 12u) *reinterpret_cast<uint32_t*>(h + 2) = b;
        if ((r & 3u) == 1u) h[0] = (uint16_t)a;
        if ((r & 3u) == 2u) h[1] = (uint16_t)(a >> 16);
        if ((r & 12u) == 4u) h[2] = (uint16_t)b;
        if ((r & 12u) == 8u) h[3] = (uint16_t)(b >> 16);
    }
};
template <> struct Unit<float> {
    static constexpr int V = 4, P = 2;
    float4 r;
    __device__ __forceinline__ void load(const float* p) { r = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void load_stream(const float* p) { r = __ldcs(reinterpret_cast<const float4*>(p)); }
    __device__ __forceinline__ void zero() { r = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    __device__ __forceinline__ f32x2 at(int i) const { return i == 0 ? two(r.x, r.y) : two(r.z, r.w); }
    __device__ __forceinline__ void keep(uint32_t ok) {
        r = make_float4((ok & 1u) ? r.x : 0.0f, (ok & 2u) ? r.y : 0.0f, (ok & 4u) ? r.z : 0.0f, (ok & 8u) ? r.w : 0.0f);
    }
    __device__ __forceinline__ void load_some(const float* p, uint32_t ok) {
        r = make_float4((ok & 1u) ? p[0] : 0.0f, (ok & 2u) ? p[1] : 0.0f, (ok & 4u) ? p[2] : 0.0f, (ok & 8u) ? p[3] : 0.0f);
    }
    __device__ static __forceinline__ void store(float* p, const f32x2 (&f)[2]) {
        const float2 a = parts(f[0]), b = parts(f[1]);
        __stcs(reinterpret_cast<float4*>(p), make_float4(a.x, a.y, b.x, b.y));
    }
    __device__ static __forceinline__ void store_some(float* p, const f32x2 (&f)[2], uint32_t ok) {
        const float2 a = parts(f[0]), b = parts(f[1]);
        if (ok & 1u) p[0] = a.x;
        if (ok & 2u) p[1] = a.y;
        if (ok & 4u) p[2] = b.x;
        if (ok & 8u) p[3] = b.y;
    }
};

// The columns of a thread's NV units of every row it meets: units first, first + step, .. of the row, counted
// from the aligned address at or before its start, `off` elements before it. Rows whose distance is a multiple
// of V have the same off, and a thread meets only such rows, so that a width that is no multiple of V (kRagged)
// differs only in the edge units: bits of `ok` say which elements of a unit are the row's.
template <typename T, int NV, bool kRagged> struct Columns {
    static constexpr int V = Unit<T>::V, P = V / 2;
    static constexpr uint32_t kAll = (1u << V) - 1u;
    int first, step, off, units;
    uint32_t bits[kRagged ? NV : 1];
    __device__ __forceinline__ void init(int first_, int step_, int64_t row, int width) {
        first = first_;
        step = step_;
        off = kRagged ? (int)((row * width) % V) : 0;
        units = (off + width + V - 1) / V;
        if constexpr (kRagged)
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                bits[k] = 0u;
#pragma unroll
                for (int e = 0; e < V; ++e) bits[k] |= (unsigned)(column(k) + e) < (unsigned)width ? 1u << e : 0u;
            }
    }
    __device__ __forceinline__ int unit(int k) const { return first + step * k; }
    __device__ __forceinline__ bool in(int k) const { return unit(k) < units; }
    __device__ __forceinline__ int column(int k) const { return unit(k) * V - off; }    // of its element 0
    __device__ __forceinline__ uint32_t ok(int k) const { return kRagged ? bits[kRagged ? k : 0] : kAll; }
    __device__ __forceinline__ bool whole(int k) const { return !kRagged || ok(k) == kAll; }
    // row: element 0 of the row; left: elements from there to the tensor's end. The elements that are not the
    // row's are still to be taken out (keep), when no more loads wait to be issued.
    __device__ __forceinline__ void load(Unit<T>& u, int k, const T* row, int64_t left) const {
        if (kRagged && column(k) + V > left) u.load_some(row + column(k), ok(k));
        else u.load_stream(row + column(k));
    }
    __device__ __forceinline__ void keep(Unit<T>& u, int k) const {
        if (!whole(k)) u.keep(ok(k));
    }
    __device__ __forceinline__ void store(T* row, int k, const f32x2 (&f)[P]) const {
        if (whole(k)) {
            Unit<T>::store(row + column(k), f);
        } else {
            Unit<T>::store_some(row + column(k), f, ok(k));
        }
    }
    // the same for fp32 sums of the columns, at any alignment
    __device__ __forceinline__ void leave(float* sums, int k, const f32x2 (&f)[P]) const {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float2 x = parts(f[i]);
            if ((ok(k) >> (2 * i)) & 1u) sums[column(k) + 2 * i] = x.x;
            if ((ok(k) >> (2 * i + 1)) & 1u) sums[column(k) + 2 * i + 1] = x.y;
        }
    }
    // adds (x - mu)^2 of the unit's elements that are the row's to a pair of sums
    __device__ __forceinline__ void squares(f32x2& s, const Unit<T>& u, int k, f32x2 minus_mu) const {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            f32x2 d = add2(u.at(i), minus_mu);
            if constexpr (kRagged) {
                const float2 x = parts(d);
                d = two((ok(k) >> (2 * i)) & 1u ? x.x : 0.0f, (ok(k) >> (2 * i + 1)) & 1u ? x.y : 0.0f);
            }
            s = fma2(d, d, s);
        }
    }
    // the parameters of unit k, `other` without them
    __device__ __forceinline__ void params(const float* p, int k, float other, f32x2 (&f)[P]) const {
        if (!p || !in(k)) {
#pragma unroll
            for (int i = 0; i < P; ++i) f[i] = two(other, other);
        } else if constexpr (kRagged) {
#pragma unroll
            for (int i = 0; i < P; ++i)
                f[i] = two((ok(k) >> (2 * i)) & 1u ? __ldg(p + column(k) + 2 * i) : other,
                           (ok(k) >> (2 * i + 1)) & 1u ? __ldg(p + column(k) + 2 * i + 1) : other);
        } else {
#pragma unroll
            for (int i = 0; i < P; i += 2) {
                const float4 x = __ldg(reinterpret_cast<const float4*>(p + column(k) + 2 * i));
                f[i] = two(x.x, x.y);
                f[i + 1] = two(x.z, x.w);
            }
        }
    }
};

// A thread's columns are its own for all rows, so their parameters stay in registers, up to 24 columns
// (they are as long as two or four bf16 rows: fetched for every row, 96 KB of them at a width of 12288
// came from L2 each time and held the forward at 3.1 of 6.7 TB/s).
template <typename T, int NV, bool kRagged> struct Params {
    static constexpr int P = Unit<T>::P;
    static constexpr bool kept = NV * Unit<T>::V <= 24;
    const float* p;
    float other;
    f32x2 f[kept ? NV : 1][P];
    __device__ __forceinline__ void init(const Columns<T, NV, kRagged>& c, const float* from, float without) {
        p = from;
        other = without;
        if constexpr (kept)
#pragma unroll
            for (int k = 0; k < NV; ++k) c.params(p, k, other, f[k]);
    }
    __device__ __forceinline__ void at(const Columns<T, NV, kRagged>& c, int k, f32x2 (&o)[P]) const {
        if constexpr (kept)
#pragma unroll
            for (int i = 0; i < P; ++i) o[i] = f[k][i];
        else c.params(p, k, other, o);
    }
};

__device__ __forceinline__ float both(f32x2 x) {
    const float2 p = parts(x);
    return p.x + p.y;
}
// y of a pair, and dx of a pair: xh and a = dy w, then rstd (a - s1 - xh s2)
__device__ __forceinline__ f32x2 norm_y(f32x2 x, f32x2 minus_mu, f32x2 rs, f32x2 w, f32x2 b) { return fma2(mul2(add2(x, minus_mu), rs), w, b); }
__device__ __forceinline__ f32x2 norm_dx(f32x2 xh, f32x2 a, f32x2 rs, f32x2 minus_s1, f32x2 minus_s2) {
    return mul2(rs, fma2(xh, minus_s2, add2(a, minus_s1)));
}

// ---------------------------------------------------------------------------------- narrow
// Lanes lpr * s .. lpr * (s + 1) - 1 of a warp hold row s of its 32 / lpr rows, lane l of them units l and l + lpr
// (with one unit a lane and twice the lanes the sums' shuffles cost as much for half the rows, which took 13% to 30%
// more: backward 131072 x 128 bf16 28 instead of 24.7 us, forward 161374 x 128 fp32 39 instead of 30). A block has eight warps, and the rows of a
// step lie a multiple of eight from those of the step before.
constexpr int kNarrowNV = 2;
__device__ __forceinline__ float lanes_sum(float x, int lpr) {
    for (int o = lpr >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// rows in flight of the forward, by a thread's columns, and blocks on an SM (32768 x 512 bf16 17.9 us with (1, 6), 20.7 with
// (2, 4); 32768 x 501 35 and 30)
__host__ __device__ constexpr int fwd_rows(int columns, bool ragged) { return columns <= 8 || ragged ? 2 : 1; }
template <typename T, int NV, bool kRagged>
__global__ void __launch_bounds__(kThreads)
    norm_fwd_narrow_kernel(const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ b, T* __restrict__ y,
                           float* __restrict__ mean, float* __restrict__ rstd, int64_t rows, int width, int lpr, float eps) {
    constexpr int P = Unit<T>::P, R = fwd_rows(2 * P * NV, kRagged);
    const int lane = threadIdx.x & 31, sub = lane / lpr, l = lane % lpr, rpw = 32 / lpr;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 32) * rpw;
    const int64_t first = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * rpw;
    const float inv = 1.0f / (float)width;
    Columns<T, NV, kRagged> c;
    c.init(l, lpr, first + sub, width);
    Params<T, NV, kRagged> pw, pb;
    pw.init(c, w, 1.0f);
    pb.init(c, b, 0.0f);
    for (int64_t r0 = first; r0 < rows; r0 += R * step) {
        Unit<T> u[R][NV];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int64_t r = r0 + q * step + sub;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (r < rows && c.in(k)) c.load(u[q][k], k, x + r * width, (rows - r) * width);
                else u[q][k].zero();
            }
        }
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int64_t r = r0 + q * step + sub;
            f32x2 s = 0ull;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                c.keep(u[q][k], k);
#pragma unroll
                for (int i = 0; i < P; ++i) s = add2(s, u[q][k].at(i));
            }
            const float mu = lanes_sum(both(s), lpr) * inv;
            const f32x2 minus_mu = two(-mu, -mu);
            s = 0ull;
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (c.in(k)) c.squares(s, u[q][k], k, minus_mu);
            const float rs = rsqrtf(lanes_sum(both(s), lpr) * inv + eps);
            const f32x2 rs2 = two(rs, rs);
            if (r >= rows) continue;
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (c.in(k)) {
                    f32x2 wv[P], bv[P], o[P];
                    pw.at(c, k, wv);
                    pb.at(c, k, bv);
#pragma unroll
                    for (int i = 0; i < P; ++i) o[i] = norm_y(u[q][k].at(i), minus_mu, rs2, wv[i], bv[i]);
                    c.store(y + r * width, k, o);
                }
            if (l == 0) {
                if (mean) mean[r] = mu;
                if (rstd) rstd[r] = rs;
            }
        }
    }
}

// rows in flight of the backward, two blocks on an SM (65536 x 256 fp32 35 us, with two rows 38; 32768 x 512 bf16 25 us,
// with one 33; three blocks of two rows 40)
__host__ __device__ constexpr int bwd_narrow_rows(int columns) { return columns <= 8 ? 3 : 2; }
constexpr int kNarrowBlocks = 2;
template <typename T, int NV, bool kRagged>
__global__ void __launch_bounds__(kThreads, kNarrowBlocks)
    norm_bwd_narrow_kernel(const T* __restrict__ x, const T* __restrict__ dy, const float* __restrict__ w,
                           const float* __restrict__ mean, const float* __restrict__ rstd, T* __restrict__ dx,
                           float* __restrict__ part, int64_t rows, int width, int lpr) {
    constexpr int P = Unit<T>::P, R = bwd_narrow_rows(2 * P * NV);
    extern __shared__ float acc[];   // [warps, or warps * rpw][2][width]
    grid_launch_next();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / lpr, l = lane % lpr, rpw = 32 / lpr;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 32) * rpw;
    const int64_t first = ((int64_t)blockIdx.x * (kThreads / 32) + warp) * rpw;
    const float inv = 1.0f / (float)width;
    Columns<T, NV, kRagged> c;
    c.init(l, lpr, first + sub, width);
    f32x2 wv[NV][P], dw[NV][P], db[NV][P];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        c.params(w, k, 1.0f, wv[k]);
#pragma unroll
        for (int i = 0; i < P; ++i) dw[k][i] = db[k][i] = 0ull;
    }
    for (int64_t r0 = first; r0 < rows; r0 += R * step) {
        Unit<T> ux[R][NV], ug[R][NV];
        float mu[R], rs[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int64_t r = r0 + q * step + sub;
            const bool in = r < rows;
            mu[q] = in ? mean[r] : 0.0f;
            rs[q] = in ? rstd[r] : 0.0f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (in && c.in(k)) {
                    c.load(ux[q][k], k, x + r * width, (rows - r) * width);
                    c.load(ug[q][k], k, dy + r * width, (rows - r) * width);
                } else {
                    ux[q][k].zero();
                    ug[q][k].zero();
                }
            }
        }
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int64_t r = r0 + q * step + sub;
            f32x2 s1 = 0ull, s2 = 0ull;
            const f32x2 minus_mu = two(-mu[q], -mu[q]), rs2 = two(rs[q], rs[q]);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                c.keep(ux[q][k], k);
                c.keep(ug[q][k], k);   // zero where the element is not the row's: it adds nothing
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const f32x2 g = ug[q][k].at(i), h = mul2(add2(ux[q][k].at(i), minus_mu), rs2), a = mul2(g, wv[k][i]);
                    s1 = add2(s1, a);
                    s2 = fma2(a, h, s2);
                    dw[k][i] = fma2(g, h, dw[k][i]);
                    db[k][i] = add2(db[k][i], g);
                }
            }
            const float t1 = -lanes_sum(both(s1), lpr) * inv, t2 = -lanes_sum(both(s2), lpr) * inv;
            if (r < rows)
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    if (c.in(k)) {
                        f32x2 o[P];
#pragma unroll
                        for (int i = 0; i < P; ++i)
                            o[i] = norm_dx(mul2(add2(ux[q][k].at(i), minus_mu), rs2), mul2(ug[q][k].at(i), wv[k][i]), rs2, two(t1, t1), two(t2, t2));
                        c.store(dx + r * width, k, o);
                    }
        }
    }
    if (!part) return;
    // The sums of the warp's rows, of the block's warps in order. (Rows of a warp that start at different places
    // have different columns in a lane.)
    int at = warp * rpw + sub, n = kThreads / 32 * rpw;
    if constexpr (!kRagged) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < P; ++i)
                for (int o = lpr; o < 32; o <<= 1) {
                    dw[k][i] = add2(dw[k][i], __shfl_xor_sync(0xffffffffu, dw[k][i], o));
                    db[k][i] = add2(db[k][i], __shfl_xor_sync(0xffffffffu, db[k][i], o));
                }
        at = warp;
        n = kThreads / 32;
    }
    if (kRagged || sub == 0)
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (c.in(k)) {
                c.leave(acc + (size_t)(2 * at) * width, k, dw[k]);
                c.leave(acc + (size_t)(2 * at + 1) * width, k, db[k]);
            }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * width; i += kThreads) {
        float s = 0.0f;
        for (int j = 0; j < n; ++j) s += acc[(size_t)2 * j * width + i];
        part[(size_t)blockIdx.x * 2 * width + i] = s;
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
// rows at a time of the backward, by a thread's columns: 4099 x 4096 fp32 (8 columns) 41 us, 45 with one;
// 8192 x 4096 bf16 (16 columns) 54 us with one, 57 with two
__host__ __device__ constexpr int bwd_rows(int columns) { return columns <= 8 ? 2 : 1; }

// Registers of a thread in the forward (inputs 1) and the backward (2), by its units and columns: fewer leave room for more
// rows on an SM, and too few spill (forward 8192 x 4097 bf16 46 us with 96, 54 with 80, 67 with 112; 8192 x 4096 bf16 29.5
// with 80, 31.5 with 96; backward 16384 x 1024 bf16 32.5 with 96, 35.7 with 112; 4099 x 4096 fp32 41 with 112, 51 with 80).
__host__ __device__ constexpr int wide_regs(int inputs, int nv, int columns, bool ragged) {
    return inputs == 1 ? (columns <= 8 ? 64 : columns < 16 || (columns == 16 && !ragged) ? 80 : columns == 16 ? 96 : 128)
                       : (columns <= 8 ? (nv == 1 ? 96 : 112) : 128);
}

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
};
// unit k of a row from shared memory, or from global memory past the copied part
template <typename T, int NV, bool kRagged, int R>
__device__ __forceinline__ void take(Unit<T>& u, const Rows<R>& m, const Columns<T, NV, kRagged>& c, int k, const uint8_t* slot,
                                     const T* row, int64_t r) {
    if (kRagged && (size_t)r * m.row_bytes + (size_t)(c.column(k) + Unit<T>::V) * sizeof(T) > m.most) {
        u.load_some(row + c.column(k), c.ok(k));
    } else {
        u.load(reinterpret_cast<const T*>(slot + 16 * c.unit(k)));
        if (!c.whole(k)) u.keep(c.ok(k));
    }
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
// arithmetic runs in the other's waits: one row at a time took 81 instead of 72 us at 8192 x 12288); thread t
// holds units t, t + blockDim.x, .. A copy that has not arrived after 2 s leaves NaN in its rows' outputs
// (there is no workspace to report it in).
template <typename T, int NV, bool kRagged>
__global__ void __maxnreg__(wide_regs(1, NV, NV * Unit<T>::V, kRagged))
    norm_fwd_wide_kernel(const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ b, T* __restrict__ y,
                         float* __restrict__ mean, float* __restrict__ rstd, int64_t rows, int width, int pitch, int stages,
                         float eps) {
    constexpr int R = 2, P = Unit<T>::P;
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
    Columns<T, NV, kRagged> c;
    c.init(t, nt, blockIdx.x, width);
    Params<T, NV, kRagged> pw, pb;
    pw.init(c, w, 1.0f);
    pb.init(c, b, 0.0f);
    __syncthreads();
    int stage = 0;
    uint32_t phase = 0;
    for (int64_t r = blockIdx.x; r < rows; r += step) {
        const bool ok = mbar_wait(&m.full[stage], phase);
        Unit<T> u[R][NV];
        f32x2 s[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int64_t rq = r + q * m.stride;
            s[q] = 0ull;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (c.in(k) && rq < rows) take(u[q][k], m, c, k, m.slot(stage, 0, q), x + rq * width, rq);
                else u[q][k].zero();
#pragma unroll
                for (int i = 0; i < P; ++i) s[q] = add2(s[q], u[q][k].at(i));
            }
        }
        const float2 mu2 = block_sums(ok ? both(s[0]) : __int_as_float(0x7fffffff), ok ? both(s[1]) : __int_as_float(0x7fffffff), buf[0]);
        const float mu[R] = {mu2.x * inv, mu2.y * inv};
        const f32x2 minus_mu[R] = {two(-mu[0], -mu[0]), two(-mu[1], -mu[1])};
        // every thread has its part of the rows in registers: the stage takes later ones
        const int64_t next = r + stages * step;
        if (t == 0 && next < rows) m.issue(next, stage, x, nullptr);
#pragma unroll
        for (int q = 0; q < R; ++q) {
            s[q] = 0ull;
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (c.in(k)) c.squares(s[q], u[q][k], k, minus_mu[q]);
        }
        const float2 var = block_sums(both(s[0]), both(s[1]), buf[1]);
        const float rs[R] = {rsqrtf(var.x * inv + eps), rsqrtf(var.y * inv + eps)};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (c.in(k)) {
                f32x2 wv[P], bv[P], o[P];
                pw.at(c, k, wv);
                pb.at(c, k, bv);
#pragma unroll
                for (int q = 0; q < R; ++q) {
                    const int64_t rq = r + q * m.stride;
#pragma unroll
                    for (int i = 0; i < P; ++i) o[i] = norm_y(u[q][k].at(i), minus_mu[q], two(rs[q], rs[q]), wv[i], bv[i]);
                    if (rq < rows) c.store(y + rq * width, k, o);
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

// The same for the backward, with dw and db of a thread's columns in registers; one or two rows at a time (bwd_rows).
template <typename T, int NV, bool kRagged>
__global__ void __maxnreg__(wide_regs(2, NV, NV * Unit<T>::V, kRagged))
    norm_bwd_wide_kernel(const T* __restrict__ x, const T* __restrict__ dy, const float* __restrict__ w,
                         const float* __restrict__ mean, const float* __restrict__ rstd, T* __restrict__ dx,
                         float* __restrict__ part, int64_t rows, int width, int pitch, int stages) {
    constexpr int P = Unit<T>::P, R = bwd_rows(2 * P * NV);
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
    f32x2 dw[NV][P], db[NV][P];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < P; ++i) dw[k][i] = db[k][i] = 0ull;
    Columns<T, NV, kRagged> c;
    c.init(t, nt, blockIdx.x, width);
    Params<T, NV, kRagged> pw;
    pw.init(c, w, 1.0f);
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
        f32x2 minus_mu[R], rs[R], s1[R], s2[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            minus_mu[q] = two(-mu_next[q], -mu_next[q]);
            rs[q] = two(rs_next[q], rs_next[q]);
            s1[q] = s2[q] = 0ull;
        }
        fetch(r + step);
        const bool ok = mbar_wait(&m.full[stage], phase);
        Unit<T> ux[R][NV], ug[R][NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            f32x2 wv[P];
            if (c.in(k)) pw.at(c, k, wv);
#pragma unroll
            for (int q = 0; q < R; ++q) {
                const int64_t rq = r + q * m.stride;
                if (c.in(k) && rq < rows) {
                    take(ux[q][k], m, c, k, m.slot(stage, 0, q), x + rq * width, rq);
                    take(ug[q][k], m, c, k, m.slot(stage, 1, q), dy + rq * width, rq);
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        const f32x2 g = ug[q][k].at(i), h = mul2(add2(ux[q][k].at(i), minus_mu[q]), rs[q]), a = mul2(g, wv[i]);
                        s1[q] = add2(s1[q], a);
                        s2[q] = fma2(a, h, s2[q]);
                        dw[k][i] = fma2(g, h, dw[k][i]);
                        db[k][i] = add2(db[k][i], g);
                    }
                }
            }
        }
        // one barrier for the sums of all rows of the step
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const float2 p = warp_sums(ok ? both(s1[q]) : __int_as_float(0x7fffffff), both(s2[q]));
            if ((t & 31) == 0) buf[turn][q][t >> 5] = p;
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const float2 p = sum_of(buf[turn][q]);
            s1[q] = two(-p.x * inv, -p.x * inv);
            s2[q] = two(-p.y * inv, -p.y * inv);
        }
        turn ^= 1;
        const int64_t next = r + stages * step;
        if (t == 0 && next < rows) m.issue(next, stage, x, dy);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (c.in(k)) {
                f32x2 wv[P], o[P];
                pw.at(c, k, wv);
#pragma unroll
                for (int q = 0; q < R; ++q) {
                    const int64_t rq = r + q * m.stride;
#pragma unroll
                    for (int i = 0; i < P; ++i)
                        o[i] = norm_dx(mul2(add2(ux[q][k].at(i), minus_mu[q]), rs[q]), mul2(ug[q][k].at(i), wv[i]), rs[q], s1[q], s2[q]);
                    if (rq < rows) c.store(dx + rq * width, k, o);
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
        if (c.in(k)) {
            c.leave(part + (size_t)blockIdx.x * 2 * width, k, dw[k]);
            c.leave(part + ((size_t)blockIdx.x * 2 + 1) * width, k, db[k]);
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
// then the groups in order. 5 us; launched under the kernel before it (4099 x 4096 fp32 in all 41 us, 44 without).
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

constexpr int kMostParts = 4 * kSMs;   // blocks whose sums of dw and db are kept
constexpr size_t kSharedOfSM = 216 * 1024;   // for the rows of the wide form's blocks; 1 KB of each block's share is left free

// Which form a width takes, and its launch.
struct Form {
    int units, lpr, nv;      // most units of a row; lpr: lanes of a row (narrow), 0: wide or any; units a thread (wide)
    bool ragged, wide;
    int threads, pitch, stages, per_sm;
    size_t smem;
};
Form form_of(long long width, size_t size, int inputs) {
    Form f{};
    const int v = (int)(16 / size);
    f.ragged = width % v != 0;
    f.units = (int)((width + (f.ragged ? v - 1 : 0) + v - 1) / v);
    if (f.units <= kNarrowUnits) {
        f.lpr = 1;
        while (kNarrowNV * f.lpr < f.units) f.lpr *= 2;
        return f;
    }
    if (f.units > kWideMost / v) return f;   // (a row of that many columns spans one unit more where it starts inside one)
    f.wide = true;
    f.pitch = (int)((width * size + 31) / 16 * 16);
    // Two units a thread and small blocks, so that many rows are in flight; more units where 512 threads do not hold
    // the row; one in the backward of short rows, whose blocks are limited by kMostParts (20000 x 777 bf16 43 us,
    // 54 with two).
    f.nv = inputs == 2 && f.units <= 128 ? 1 : 2;
    while (f.units > f.nv * 512) f.nv = f.nv == 4 ? 8 : f.nv + 1;
    f.threads = ((f.units + f.nv - 1) / f.nv + 31) / 32 * 32;
    // warps that an SM's registers hold, in four quarters
    const int fit = 4 * (65536 / 4 / (32 * wide_regs(inputs, f.nv, f.nv * v, f.ragged))) / (f.threads / 32);
    f.per_sm = std::min(std::max(fit, 1), inputs == 1 ? 16 : kMostParts / kSMs);
    const int stage = f.pitch * inputs * (inputs == 1 ? 2 : bwd_rows(f.nv * v));
    // up to four steps ahead, within the SM's shared memory; fewer blocks rather than none ahead
    for (;; --f.per_sm) {
        f.stages = (int)((kSharedOfSM / f.per_sm - 1024 - 64) / stage);
        if (f.stages >= 2 || f.per_sm == 1) break;
    }
    f.stages = std::clamp(f.stages, 1, 4);
    f.smem = 64 + (size_t)stage * f.stages;
    return f;
}

// Allows a wide kernel as much shared memory as form_of can ask for, once for each device (`done` is the kernel's own): the
// limit is the kernel's, not the launch's, and a call that set it to its own size could take it from under a launch
// of another thread.
kda_status allow_shared(const void* kernel, std::atomic<uint64_t>& done, const char* where) {
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return launched(where);
    const uint64_t bit = device < 64 ? uint64_t(1) << device : 0;
    if (done.load(std::memory_order_relaxed) & bit) return KDA_OK;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kSharedOfSM - 1024)) != cudaSuccess) return launched(where);
    done.fetch_or(bit, std::memory_order_relaxed);
    return KDA_OK;
}

unsigned blocks(long long rows, long long most) { return (unsigned)(rows < most ? rows : most); }

template <typename T, int NV, bool kRagged>
kda_status fwd_wide(const Form& f, long long rows, int width, float eps, const T* x, const float* w, const float* b, T* y,
                    float* mean, float* rstd, cudaStream_t s) {
    auto k = norm_fwd_wide_kernel<T, NV, kRagged>;
    static std::atomic<uint64_t> allowed{0};
    const kda_status st = allow_shared(reinterpret_cast<const void*>(k), allowed, "kda_layernorm_fwd");
    if (st != KDA_OK) return st;
    k<<<blocks(rows, (long long)kSMs * f.per_sm), f.threads, f.smem, s>>>(x, w, b, y, mean, rstd, rows, width, f.pitch, f.stages, eps);
    return launched("kda_layernorm_fwd launch");
}
template <typename T, int NV, bool kRagged>
kda_status fwd_narrow(const Form& f, long long rows, int width, float eps, const T* x, const float* w, const float* b, T* y,
                      float* mean, float* rstd, cudaStream_t s) {
    const long long rpb = (long long)(kThreads / 32) * (32 / f.lpr);
    constexpr int per_sm = fwd_rows(Unit<T>::V * NV, kRagged) == 2 ? 4 : 6;
    norm_fwd_narrow_kernel<T, NV, kRagged><<<blocks((rows + rpb - 1) / rpb, per_sm * kSMs), kThreads, 0, s>>>(
        x, w, b, y, mean, rstd, rows, width, f.lpr, eps);
    return launched("kda_layernorm_fwd launch");
}
template <typename T, bool kRagged>
kda_status fwd(const Form& f, long long rows, int width, float eps, const void* xv, const float* w, const float* b, void* yv,
               float* mean, float* rstd, cudaStream_t s) {
    const T* x = static_cast<const T*>(xv);
    T* y = static_cast<T*>(yv);
#define KDA_NORM(fn, n) return fn<T, n, kRagged>(f, rows, width, eps, x, w, b, y, mean, rstd, s)
    if (f.lpr) KDA_NORM(fwd_narrow, kNarrowNV);
    if (f.wide) {
        if (f.nv == 2) KDA_NORM(fwd_wide, 2);
        if (f.nv == 3) KDA_NORM(fwd_wide, 3);
        if (f.nv == 4) KDA_NORM(fwd_wide, 4);
        if constexpr (sizeof(T) == 4) KDA_NORM(fwd_wide, 8);
    }
#undef KDA_NORM
    norm_fwd_any_kernel<T><<<blocks(rows, 1 << 30), kThreads, 0, s>>>(x, w, b, y, mean, rstd, rows, width, eps);
    return launched("kda_layernorm_fwd launch");
}

template <typename T, int NV, bool kRagged>
kda_status bwd_wide(const Form& f, long long rows, int width, const T* x, const T* dy, const float* w, const float* mean,
                    const float* rstd, T* dx, float* part, int* parts, cudaStream_t s) {
    auto k = norm_bwd_wide_kernel<T, NV, kRagged>;
    static std::atomic<uint64_t> allowed{0};
    const kda_status st = allow_shared(reinterpret_cast<const void*>(k), allowed, "kda_layernorm_bwd");
    if (st != KDA_OK) return st;
    *parts = (int)blocks(rows, (long long)kSMs * f.per_sm);
    k<<<*parts, f.threads, f.smem, s>>>(x, dy, w, mean, rstd, dx, part, rows, width, f.pitch, f.stages);
    return launched("kda_layernorm_bwd launch");
}
template <typename T, int NV, bool kRagged>
kda_status bwd_narrow(const Form& f, long long rows, int width, const T* x, const T* dy, const float* w, const float* mean,
                      const float* rstd, T* dx, float* part, int* parts, cudaStream_t s) {
    const int rpw = 32 / f.lpr;
    const long long rpb = (long long)(kThreads / 32) * rpw;
    const size_t smem = (size_t)rpb * 2 * width * sizeof(float);
    *parts = (int)blocks((rows + rpb - 1) / rpb, kNarrowBlocks * kSMs);   // as many as are resident
    norm_bwd_narrow_kernel<T, NV, kRagged><<<*parts, kThreads, smem, s>>>(x, dy, w, mean, rstd, dx, part, rows, width, f.lpr);
    return launched("kda_layernorm_bwd launch");
}
// dx and, to part where it is given, the sums of `parts` blocks
template <typename T, bool kRagged>
kda_status bwd(const Form& f, long long rows, int width, const void* xv, const void* dyv, const float* w, const float* mean,
               const float* rstd, void* dxv, float* part, int* parts, cudaStream_t s) {
    const T *x = static_cast<const T*>(xv), *dy = static_cast<const T*>(dyv);
    T* dx = static_cast<T*>(dxv);
#define KDA_NORM(fn, n) return fn<T, n, kRagged>(f, rows, width, x, dy, w, mean, rstd, dx, part, parts, s)
    if (f.lpr) KDA_NORM(bwd_narrow, kNarrowNV);
    if (f.wide) {
        if (f.nv == 1) KDA_NORM(bwd_wide, 1);
        if (f.nv == 2) KDA_NORM(bwd_wide, 2);
        if (f.nv == 3) KDA_NORM(bwd_wide, 3);
        if (f.nv == 4) KDA_NORM(bwd_wide, 4);
        if constexpr (sizeof(T) == 4) KDA_NORM(bwd_wide, 8);
    }
#undef KDA_NORM
    *parts = (int)blocks(rows, kSMs);
    if (part)   // before dx, which may take the place of x or dy
        norm_dw_any_kernel<T><<<dim3((unsigned)((width + kThreads - 1) / kThreads), (unsigned)*parts), kThreads, 0, s>>>(
            x, dy, mean, rstd, part, rows, width);
    norm_dx_any_kernel<T><<<blocks(rows, 1 << 30), kThreads, 0, s>>>(x, dy, w, mean, rstd, dx, rows, width);
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
    const Form f = form_of(width, dtype == KDA_BF16 ? 2 : 4, 1);
    auto run = dtype == KDA_BF16 ? (f.ragged ? fwd<uint16_t, true> : fwd<uint16_t, false>) : (f.ragged ? fwd<float, true> : fwd<float, false>);
    return run(f, rows, (int)width, eps, x, weight, bias, y, mean, rstd, s);
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
        const Form f = form_of(width, dtype == KDA_BF16 ? 2 : 4, 2);
        auto run = dtype == KDA_BF16 ? (f.ragged ? bwd<uint16_t, true> : bwd<uint16_t, false>) : (f.ragged ? bwd<float, true> : bwd<float, false>);
        const kda_status st = run(f, rows, (int)width, x, dy, weight, mean, rstd, dx, part, &parts, s);
        if (st != KDA_OK) return st;
    }
    if (sums)
        launch_kernel(norm_reduce_kernel, dim3((unsigned)((width + 31) / 32), 2), dim3(32, 32), 0, s, parts > 0,
                      static_cast<const float*>(workspace), parts, (int)width, dweight, dbias);
    return launched("kda_layernorm_bwd launch");
}
