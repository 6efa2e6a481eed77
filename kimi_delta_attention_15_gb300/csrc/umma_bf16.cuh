// Further building blocks (see umma.cuh) of the bf16 kernels: tensor loads and stores, waits that sleep,
// tensor-memory stores, kind::f16 MMAs with bf16 operands and their tiles, overlapped launches.
#pragma once
#include <utility>
#include "umma.cuh"

namespace kda {

// ---------------------------------------------------------------- mbarrier
// mbar_wait for kernels whose waiting warps share an SM's issue slots with working ones: the thread may
// sleep in the hardware for up to 20 us at a time and is woken when the phase completes.
__device__ __forceinline__ bool mbar_try_wait_asleep(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_asleep(uint64_t* bar, uint32_t parity, uint64_t limit_ns = kWaitLimitNs) {
    if (mbar_try_wait_asleep(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        if (mbar_try_wait_asleep(bar, parity)) return true;
        if (globaltimer_ns() - t0 > limit_ns) return false;
    }
}

// --------------------------------------------------------- tensor (TMA) copies
// A box of a 3-D tensor (its map in kernel parameter space) -> shared, completion counted in bytes
// on an mbarrier. The innermost coordinate x starts on a 16-byte boundary; rows out of range,
// negative ones too, arrive as zeros.
__device__ __forceinline__ void tma_load_3d(void* dst, const void* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// The same box into L2 only.
__device__ __forceinline__ void tma_prefetch_3d(const void* map, int x, int y, int z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
// shared -> a box of a 3-D tensor, tracked by bulk async-groups. No coordinate may be negative.
__device__ __forceinline__ void tma_store_3d(const void* src, const void* map, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
                 "r"(x), "r"(y), "r"(z), "r"(smem_u32(src))
                 : "memory");
}

// ------------------------------------------------------------------ TMEM
// 32 lanes x 16 consecutive columns; the same rule for v until tmem_wait_st_all
__device__ __forceinline__ void tmem_st16_issue(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
// 16 lanes (the first or second half of the warp's 32, by the address) x 16 consecutive columns from
// ldmatrix fragments: register 2 m + e of thread t holds column 4 m + t % 4 of lane 8 e + t / 4
__device__ __forceinline__ void tmem_st_frag_issue(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
        "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
        : "memory");
}
// four 8x8 matrices of 16-bit values, transposed: lanes 8 i .. 8 i + 7 give the row addresses of matrix
// i; register i of thread t holds elements (2 (t % 4), t / 4) and (2 (t % 4) + 1, t / 4) of it
__device__ __forceinline__ void ldmatrix4_trans(uint32_t saddr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
                 : "r"(saddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st_all() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// --------------------------------------------------------------------- MMA
// Instruction descriptor for kind::f16 with bf16 operands and fp32 accumulation.
// a_mn / b_mn: 0 = operand is K-major, 1 = MN-major.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, int a_mn, int b_mn) {
    return (1u << 4)                       // D format: f32
           | (1u << 7)                     // A format: bf16
           | (1u << 10)                    // B format: bf16
           | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}

// D[tmem] (+)= A * B^T in bf16, one instruction (K = 16). Issued by one thread.
__device__ __forceinline__ void umma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// The same with A in tensor memory: lane m holds row m, the 8 columns from a_tmem the 16 K
// values of this step, two to a column.
__device__ __forceinline__ void umma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// bf16 operand tiles of R rows x 128 columns: panels of 64 columns (128 bytes per row), each
// panel [R][64] contiguous with the same 128-byte swizzle. Byte offset of the 16-byte chunk
// (8 columns) ch = 0 .. 15 of row r:
__host__ __device__ __forceinline__ uint32_t panel_off_bf16(uint32_t r, uint32_t ch, uint32_t R) {
    return (ch >> 3) * R * 128u + r * 128u + (((ch & 7u) ^ (r & 7u)) << 4);
}
// k-step s of such a tile as an operand [MN columns][K rows] (MN-major): rows 16 s .. 16 s + 15.
// 64-column panels along MN are R * 128 bytes apart, 8-row groups along K 1024 bytes. (As a
// K-major operand, [MN rows][K columns], its step s of 16 columns has desc_kmajor's descriptor.)
__device__ __forceinline__ uint64_t desc_mnmajor_bf16(uint32_t tile_saddr, uint32_t R, uint32_t s) {
    return sdesc_sw128(tile_saddr + s * 2048u, R * 128u, 1024u);
}

// ------------------------------------------------------------- packed fp32
// two fp32 values in one 64-bit register, multiplied and added in one instruction
using f32x2 = uint64_t;
__device__ __forceinline__ f32x2 two(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ f32x2 two(uint32_t a, uint32_t b) { return two(__uint_as_float(a), __uint_as_float(b)); }
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float2 parts(f32x2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}

// ---------------------------------------------------------------- launches
// Overlap of a kernel's launch with the kernel before it (launch_kernel with `overlap`): the kernel before allows
// it to start, and it waits until that one has finished and its writes can be read. Neither does anything in a
// kernel that is launched without overlap.
__device__ __forceinline__ void grid_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A launch; with `overlap` the kernel may start before the one before it on the stream has finished, and waits for
// it (grid_wait_before) ahead of anything it reads or writes in global memory.
template <typename... P, typename... A>
inline void launch_kernel(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, bool overlap, A&&... args) {
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = block;
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    c.attrs = &at;
    c.numAttrs = overlap ? 1 : 0;
    cudaLaunchKernelEx(&c, kernel, std::forward<A>(args)...);   // an error is left for cudaGetLastError
}

}  // namespace kda
