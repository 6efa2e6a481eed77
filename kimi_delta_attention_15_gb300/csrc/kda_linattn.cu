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
#include "umma.cuh"

namespace kda {
void set_last_error_text(const char* msg);

namespace {

constexpr int LC = 128;                       // tokens of a chunk
constexpr int kSMs = 152;                     // of a GB300; one persistent CTA on each
// the cost model of the split, in chunk times of a full unit
constexpr double kStateOnly = 0.5, kUnitChunks = 1.0, kSplitChunks = 4.0;
constexpr uint32_t kTile = LC * D * 2;        // a bf16 operand tile [128][128], two 64-column panels

// One sum over tokens in the roles' names. Row i of a chunk of L rows, with the state S the
// chunk starts from (e = 1 forward, 0 reversed: a token's decay applies before or after its read):
//   out_i = out_scale (sum_{j <= i} k_scale gamma^{i-j} (q_i . k_j) v_j + gamma^{i+e} S q_i)
//   S    <- gamma^L S + sum_j k_scale gamma^{L-e-j} v_j k_j^T
struct LinJob {
    const uint16_t *q, *k, *v;   // [tokens, H / g?, 128]
    int gq, gk, gv;              // value heads that share a head of each
    uint16_t* out;               // [tokens, H, 128] bf16, or
    float* share;                // [tokens, H, 128] fp32: each value head's share of a grouped sum
    const float* s_in;           // initial state [N, H, 128, 128], may be NULL
    float* s_out;                // final state, may be NULL
    float* seg;                  // states of the segments [slots, H, 128, 128]
    int s_in_t, seg_t;           // s_in, seg are stored transposed
    int rev;                     // tokens from last to first
    int pieces;                  // bf16 parts of the decayed k in the state's sum: 2 or 3
    float k_scale, out_scale;
};

// A slot is a segment of a sequence; a sequence has one at least, an empty one too.
struct Slot {
    int64_t t0;         // first token
    int32_t len, seq;
    int32_t seg, nseg;  // its place among the sequence's segments
};

struct LinArgs {
    LinJob job[3];
    int jobs;
    int state_only;              // the segments' own states to seg, nothing else
    int first;                   // the first kernel of the call on this workspace: clears its status word
    const Slot* table;           // packed: slots and their number, written by linattn_table_kernel
    const int* slots_dev;
    int slots;                   // fixed length: nseg segments of seg_len tokens per sequence
    int nseg;
    int64_t seg_len, T;
    const float* log_decay;
    int H;
    uint8_t* ws;
};

__device__ __forceinline__ float decay_pow(float g, int n) { return n == 0 ? 1.0f : expf(g * (float)n); }

__device__ __forceinline__ Slot slot_of(const LinArgs& a, int i) {
    if (a.table) return a.table[i];
    Slot s;
    s.seq = i / a.nseg;
    s.seg = i - s.seq * a.nseg;
    s.nseg = a.nseg;
    const int64_t at = s.seg * a.seg_len, left = a.T - at;
    s.t0 = s.seq * a.T + at;
    s.len = (int32_t)(left < a.seg_len ? (left > 0 ? left : 0) : a.seg_len);
    return s;
}

struct Unit {
    const LinJob* job;
    int64_t t0;
    int len, h;
    size_t seq_state, seg_state;   // element offsets of the (sequence, head) and (slot, head) states
    const float* s_in;             // where this unit's state comes from and goes to, NULL: zero, not wanted
    float* s_out;
    int s_in_t;
};
__device__ __forceinline__ Unit unit_of(const LinArgs& a, int u) {
    const int per = a.jobs * a.H;
    const int i = u / per, r = u - i * per;
    const Slot s = slot_of(a, i);
    Unit x;
    x.job = &a.job[r / a.H];
    x.h = r % a.H;
    x.t0 = s.t0;
    x.len = s.len;
    x.seq_state = ((size_t)s.seq * a.H + x.h) * D * D;
    x.seg_state = ((size_t)i * a.H + x.h) * D * D;
    const LinJob& j = *x.job;
    const bool head = j.rev ? s.seg == s.nseg - 1 : s.seg == 0, tail = j.rev ? s.seg == 0 : s.seg == s.nseg - 1;
    if (a.state_only) {            // every segment but the last of its sequence starts from zero and leaves its sum
        x.s_in = nullptr;
        x.s_in_t = 0;
        x.s_out = tail ? nullptr : j.seg + x.seg_state;
        if (tail) x.len = 0;
    } else {
        x.s_in = head ? (j.s_in ? j.s_in + x.seq_state : nullptr) : j.seg + x.seg_state;
        x.s_in_t = head ? j.s_in_t : j.seg_t;
        x.s_out = tail && j.s_out ? j.s_out + x.seq_state : nullptr;
    }
    return x;
}
__device__ __forceinline__ int units_of(const LinArgs& a) { return (a.table ? *a.slots_dev : a.slots) * a.H * a.jobs; }
// the units of a CTA: every round of gridDim.x units in turn from the other end, so that with slots in
// order of falling length no CTA gets the longer one each time
__device__ __forceinline__ int unit_at(int round) {
    return round * (int)gridDim.x + (int)((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

struct LinSmem {
    // operand tiles (bf16 panels, 1024-byte aligned)
    uint8_t K[2][kTile];     // keys by chunk parity; once scored, overwritten with the decayed keys' high parts
    uint8_t Q[kTile];
    uint8_t V[kTile];
    uint8_t MID[kTile];      // the decayed keys' middle and low parts
    uint8_t LOW[kTile];
    uint8_t S[kTile];        // the state [v][c] the chunk starts from, rounded to bf16
    // full: operands in shared memory; qk, qs, pv, ds: MMA groups done; s, p, piece: operands written;
    // o: accumulators read. Each completes one phase per chunk. A wait names a phase by its parity, so
    // no waiter may be a whole phase behind: every wait comes before an arrival of the same thread
    // (or an MMA that needs one) on which the barrier's next phase depends.
    uint64_t full_qk, full_v, qk, qs, pv, ds, s, p, piece, o;
    uint32_t tmem;
};

// Warps 0-3: scores and outputs (thread = row of the chunk = TMEM lane). Warps 4-11: the state
// (thread = half a row) and the decayed keys. Warps 12, 13: loads. Warp 14: MMAs.
constexpr int kScoreWarps = 4, kStateWarps = 8, kLoadWarps = 2;
constexpr int kLinThreads = 32 * (kScoreWarps + kStateWarps + kLoadWarps + 1);

__device__ __forceinline__ bool wait_warp(uint64_t* bar, int n) {
    return __all_sync(0xffffffffu, mbar_wait(bar, (uint32_t)(n & 1)));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ float low_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// --- loads: cp.async, 16 bytes a thread, zeros for rows past the end of the segment
__device__ void lin_load(const LinArgs& a, LinSmem& sm, int units) {
    const int p = threadIdx.x - 32 * (kScoreWarps + kStateWarps);
    const int ch = p & 15, r0 = p >> 4;      // its 16-byte chunk, rows r0 + 4 i
    const uint32_t off[2] = {panel_off_bf16(r0, ch, LC), panel_off_bf16(r0 + 4, ch, LC)};
    auto tile = [&](uint8_t* dst, const uint16_t* base, int heads, int head, const Unit& u, int c) {
        const int64_t step = (u.job->rev ? -(int64_t)heads : (int64_t)heads) * D;
        const int left = u.len - c * LC;
        const int64_t first = u.job->rev ? u.t0 + u.len - 1 - c * LC : u.t0 + c * LC;
        const uint16_t* src0 = base + (first * heads + head) * D + ch * 8;
#pragma unroll
        for (int i = 0; i < LC / 4; ++i) {
            const int r = r0 + 4 * i;
            cp_async16_zfill(dst + off[i & 1] + (i >> 1) * 1024, r < left ? src0 + r * step : base, r < left);
        }
        cp_async_commit();
    };
    bool ok = true;
    int n = 0;
    bool have_k = false;      // this chunk's keys were requested with the chunk before
    for (int round = 0; ok; ++round) {
        const int at = unit_at(round);
        if (at >= units) break;
        const Unit u = unit_of(a, at);
        const LinJob& j = *u.job;
        const int chunks = (u.len + LC - 1) / LC;
        const int hq = a.H / j.gq, hk = a.H / j.gk, hv = a.H / j.gv;
        for (int c = 0; c < chunks; ++c, ++n) {
            // K[n & 1] was last read by the state product of chunk n - 2, which this thread waited for
            // with the V of chunk n - 1
            if (!have_k) tile(sm.K[n & 1], j.k, hk, u.h / j.gk, u, c);
            if (n > 0 && !wait_warp(&sm.qs, n - 1)) { ok = false; break; }
            if (!a.state_only) tile(sm.Q, j.q, hq, u.h / j.gq, u, c);
            cp_async_wait_all();
            fence_async_smem();
            mbar_arrive(&sm.full_qk);
            if (n > 0 && !wait_warp(&sm.ds, n - 1)) { ok = false; break; }
            tile(sm.V, j.v, hv, u.h / j.gv, u, c);
            have_k = c + 1 < chunks;
            if (have_k) tile(sm.K[(n + 1) & 1], j.k, hk, u.h / j.gk, u, c + 1);
            if (have_k) asm volatile("cp.async.wait_group 1;" ::: "memory");
            else cp_async_wait_all();
            fence_async_smem();
            mbar_arrive(&sm.full_v);
        }
    }
    cp_async_wait_all();
    if (!ok) raise_status(a.ws, KDA_ERR_TIMEOUT);
}

// --- MMAs, one thread. TMEM: scores (and their bf16 copy, two to a column), Q S^T, scores V, state sum
constexpr uint32_t kColP = 0, kColQS = 128, kColPV = 256, kColDS = 384;
__device__ void lin_mma(const LinArgs& a, LinSmem& sm, int units, uint32_t tm) {
    constexpr uint32_t kk = idesc_bf16(128, 128, 0, 0), kn = idesc_bf16(128, 128, 0, 1), mn = idesc_bf16(128, 128, 1, 1);
    const uint32_t q = smem_u32(sm.Q), v = smem_u32(sm.V), st = smem_u32(sm.S);
    const uint32_t mid = smem_u32(sm.MID), low = smem_u32(sm.LOW);
    bool ok = true;
    int n = 0;
    for (int round = 0; ok; ++round) {
        const int at = unit_at(round);
        if (at >= units) break;
        const Unit u = unit_of(a, at);
        const int chunks = (u.len + LC - 1) / LC;
        for (int c = 0; c < chunks; ++c, ++n) {
            const uint32_t ph = (uint32_t)(n & 1), k = smem_u32(sm.K[n & 1]);
            if (!(ok = mbar_wait(&sm.full_qk, ph))) break;
            tc_fence_after();
            if (!a.state_only)
                for (int s = 0; s < 8; ++s) umma_bf16(tm + kColP, desc_kmajor(q, LC, s), desc_kmajor(k, LC, s), kk, s > 0);
            umma_commit(&sm.qk);
            if (!(ok = mbar_wait(&sm.s, ph) && (n == 0 || mbar_wait(&sm.o, ph ^ 1u)))) break;
            tc_fence_after();
            if (!a.state_only && (c > 0 || u.s_in))
                for (int s = 0; s < 8; ++s) umma_bf16(tm + kColQS, desc_kmajor(q, LC, s), desc_kmajor(st, LC, s), kk, s > 0);
            umma_commit(&sm.qs);
            if (!(ok = mbar_wait(&sm.p, ph) && mbar_wait(&sm.full_v, ph))) break;
            tc_fence_after();
            if (!a.state_only)
                for (int s = 0; s < 8; ++s) umma_bf16_ta(tm + kColPV, tm + kColP + 8 * s, desc_mnmajor_bf16(v, LC, s), kn, s > 0);
            umma_commit(&sm.pv);
            if (!(ok = mbar_wait(&sm.piece, ph))) break;
            tc_fence_after();
            if (c + 1 < chunks || u.s_out) {   // small parts first: the accumulator is rounded at its size
                uint32_t acc = 0;
                if (u.job->pieces > 2)
                    for (int s = 0; s < 8; ++s, acc = 1)
                        umma_bf16(tm + kColDS, desc_mnmajor_bf16(v, LC, s), desc_mnmajor_bf16(low, LC, s), mn, acc);
                for (int s = 0; s < 8; ++s, acc = 1)
                    umma_bf16(tm + kColDS, desc_mnmajor_bf16(v, LC, s), desc_mnmajor_bf16(mid, LC, s), mn, acc);
                for (int s = 0; s < 8; ++s)
                    umma_bf16(tm + kColDS, desc_mnmajor_bf16(v, LC, s), desc_mnmajor_bf16(k, LC, s), mn, 1);
            }
            umma_commit(&sm.ds);
        }
    }
    if (!ok) {
        raise_status(a.ws, KDA_ERR_TIMEOUT);
        umma_commit(&sm.ds);                   // MMAs still in flight end before the tensor memory is freed
        mbar_wait(&sm.ds, (uint32_t)(n & 1));
    }
}

// --- scores -> decayed bf16 scores in TMEM; outputs
__device__ void lin_scores(const LinArgs& a, LinSmem& sm, int units, uint32_t tm) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = threadIdx.x;
    const uint32_t lanes = tm + ((uint32_t)(32 * warp) << 16);
    bool ok = true;
    int n = 0;
    for (int round = 0; ok; ++round) {
        const int at = unit_at(round);
        if (at >= units) break;
        const Unit u = unit_of(a, at);
        const LinJob& j = *u.job;
        const int chunks = (u.len + LC - 1) / LC;
        if (chunks == 0) continue;
        const float g = a.log_decay[u.h];
        // k_scale gamma^{row-j}: in the 32-column block left of the diagonal's by 32 m columns it is
        // gamma^{32m-31} f[j mod 32], f[x] = k_scale gamma^{lane+31-x}: no exponent is negative
        float f[32];
#pragma unroll
        for (int x = 0; x < 32; ++x) f[x] = j.k_scale * decay_pow(g, lane + 31 - x);
        const float own = j.k_scale * decay_pow(g, lane);
        const float w_state = decay_pow(g, row + (j.rev ? 0 : 1));
        for (int c = 0; c < chunks; ++c, ++n) {
            if (!(ok = wait_warp(&sm.qk, n))) break;
            tc_fence_after();
            if (!a.state_only) {
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    uint32_t w[16];
                    if (b > warp) {
#pragma unroll
                        for (int x = 0; x < 16; ++x) w[x] = 0u;
                    } else {
                        uint32_t r[32];
                        tmem_ld32_issue(lanes + kColP + 32 * b, r);
                        if (b < warp) {
                            const float base = decay_pow(g, 32 * (warp - b) - 31);
                            tmem_wait_ld(r);
#pragma unroll
                            for (int x = 0; x < 32; x += 2)
                                w[x >> 1] = pack_bf16(__uint_as_float(r[x]) * (base * f[x]), __uint_as_float(r[x + 1]) * (base * f[x + 1]));
                        } else {
                            tmem_wait_ld(r);
#pragma unroll
                            for (int x = 0; x < 32; x += 2) {
                                const float d0 = __shfl_up_sync(0xffffffffu, own, x), d1 = __shfl_up_sync(0xffffffffu, own, x + 1);
                                w[x >> 1] = pack_bf16(x <= lane ? __uint_as_float(r[x]) * d0 : 0.0f,
                                                      x + 1 <= lane ? __uint_as_float(r[x + 1]) * d1 : 0.0f);
                            }
                        }
                    }
                    tmem_st16_issue(lanes + kColP + 16 * b, w);   // behind the columns still to be read
                }
                tmem_wait_st_all();
            }
            tc_fence_before();
            mbar_arrive(&sm.p);
            if (!(ok = wait_warp(&sm.pv, n))) break;
            tc_fence_after();
            if (!a.state_only) {
                const bool carried = c > 0 || u.s_in;
                const int idx = c * LC + row;
                const int64_t t = j.rev ? u.t0 + u.len - 1 - idx : u.t0 + idx;
                const size_t at_out = (size_t)(t * a.H + u.h) * D;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    uint32_t x[32], y[32];
                    tmem_ld32_issue(lanes + kColPV + 32 * b, x);
                    if (carried) tmem_ld32_issue(lanes + kColQS + 32 * b, y);
                    tmem_wait_ld(x);
                    if (carried) {
                        tmem_after_wait(y);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            x[i] = __float_as_uint(j.out_scale * (__uint_as_float(x[i]) + w_state * __uint_as_float(y[i])));
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(j.out_scale * __uint_as_float(x[i]));
                    }
                    if (idx < u.len) {
                        if (j.share) {
#pragma unroll
                            for (int i = 0; i < 32; i += 4)
                                *reinterpret_cast<uint4*>(j.share + at_out + 32 * b + i) = make_uint4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; i += 8) {
                                uint32_t w[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) w[e] = pack_bf16(__uint_as_float(x[i + 2 * e]), __uint_as_float(x[i + 2 * e + 1]));
                                *reinterpret_cast<uint4*>(j.out + at_out + 32 * b + i) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        }
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(&sm.o);
        }
    }
    if (!ok && lane == 0) raise_status(a.ws, KDA_ERR_TIMEOUT);
}

// --- state in registers, its bf16 copy for the next chunk; decayed keys in bf16 parts
__device__ void lin_state(const LinArgs& a, LinSmem& sm, int units, uint32_t tm) {
    const int t = threadIdx.x - 32 * kScoreWarps, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = 32 * (warp & 3) + lane, half = t >> 7;       // state row, which 64 columns of it
    const uint32_t lanes = tm + ((uint32_t)(32 * (warp & 3)) << 16) + kColDS + 64 * half;
    const int ch = t & 15, r0 = t >> 4;                          // decayed keys: 16-byte chunk, rows r0 + 16 i
    const uint32_t off = panel_off_bf16(r0, ch, LC);
    bool ok = true;
    int n = 0;
    float s[64];
    auto grow = [&](float decay) {   // s = decay s + the state sum of the last chunk
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            uint32_t r[32];
            tmem_ld32_issue(lanes + 32 * b, r);
            tmem_wait_ld(r);
#pragma unroll
            for (int i = 0; i < 32; ++i) s[32 * b + i] = decay * s[32 * b + i] + __uint_as_float(r[i]);
        }
    };
    for (int round = 0; ok; ++round) {
        const int at = unit_at(round);
        if (at >= units) break;
        const Unit u = unit_of(a, at);
        const LinJob& j = *u.job;
        const int chunks = (u.len + LC - 1) / LC;
        const float g = a.log_decay[u.h];
        if (u.s_in && u.s_in_t) {
#pragma unroll
            for (int i = 0; i < 64; ++i) s[i] = u.s_in[(64 * half + i) * D + row];
        } else if (u.s_in) {
#pragma unroll
            for (int i = 0; i < 64; i += 4) {
                const float4 x = *reinterpret_cast<const float4*>(u.s_in + row * D + 64 * half + i);
                s[i] = x.x; s[i + 1] = x.y; s[i + 2] = x.z; s[i + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 64; ++i) s[i] = 0.0f;
        }
        const float whole = decay_pow(g, LC);
        const int e = j.rev ? 0 : 1;
        for (int c = 0; c < chunks; ++c, ++n) {
            if (c > 0) {
                if (!(ok = wait_warp(&sm.ds, n - 1))) break;
                tc_fence_after();
                grow(whole);
                tc_fence_before();
            }
            if (!a.state_only && (c > 0 || u.s_in)) {   // sm.S: last read by chunk n - 1, whose state product is done
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint4*>(sm.S + panel_off_bf16(row, 8 * half + i, LC)) =
                        make_uint4(pack_bf16(s[8 * i], s[8 * i + 1]), pack_bf16(s[8 * i + 2], s[8 * i + 3]),
                                   pack_bf16(s[8 * i + 4], s[8 * i + 5]), pack_bf16(s[8 * i + 6], s[8 * i + 7]));
                fence_async_smem();
            }
            // (before the arrival, without which Q of chunk n + 1 cannot complete the barrier's next phase)
            if (!(ok = wait_warp(&sm.full_qk, n))) break;
            mbar_arrive(&sm.s);
            // k_scale gamma^{L-e-j} k_j as a sum of bf16 parts: 16 significant bits in two, 24 in three
            if (!(ok = wait_warp(&sm.qk, n))) break;
            if (c + 1 < chunks || u.s_out) {
                const int L = min(LC, u.len - c * LC);
                uint8_t* const key = sm.K[n & 1];
#pragma unroll 2
                for (int i = 0; i < LC / 16; ++i) {
                    const float w = j.k_scale * decay_pow(g, max(L - e - (r0 + 16 * i), 0));
                    const uint32_t o = off + i * 2048;
                    const uint4 x = *reinterpret_cast<const uint4*>(key + o);
                    uint32_t in[4] = {x.x, x.y, x.z, x.w}, hi[4], mi[4], lo[4];
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        float p = w * low_bf16(in[d]), q = w * high_bf16(in[d]);
                        hi[d] = pack_bf16(p, q);
                        p -= low_bf16(hi[d]); q -= high_bf16(hi[d]);
                        mi[d] = pack_bf16(p, q);
                        p -= low_bf16(mi[d]); q -= high_bf16(mi[d]);
                        lo[d] = pack_bf16(p, q);
                    }
                    *reinterpret_cast<uint4*>(key + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(sm.MID + o) = make_uint4(mi[0], mi[1], mi[2], mi[3]);
                    if (j.pieces > 2) *reinterpret_cast<uint4*>(sm.LOW + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                fence_async_smem();
            }
            mbar_arrive(&sm.piece);
        }
        if (!ok) break;
        if (chunks > 0) {
            if (!(ok = wait_warp(&sm.ds, n - 1))) break;
            tc_fence_after();
            if (u.s_out) grow(decay_pow(g, u.len - (chunks - 1) * LC));
            tc_fence_before();
        }
        if (u.s_out) {
#pragma unroll
            for (int i = 0; i < 64; i += 4)
                *reinterpret_cast<float4*>(u.s_out + row * D + 64 * half + i) = make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
        }
    }
    if (!ok && lane == 0) raise_status(a.ws, KDA_ERR_TIMEOUT);
}

__global__ void __launch_bounds__(kLinThreads, 1) linattn_kernel(const __grid_constant__ LinArgs a) {
    extern __shared__ uint8_t smem_raw[];
    LinSmem& sm = *reinterpret_cast<LinSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // A fixed-length call's first kernel clears the status word here, long before any wait of
    // another CTA can give up (2 s) and write to it.
    if (a.first) {
        if (blockIdx.x == 0 && threadIdx.x == 0) *reinterpret_cast<int*>(a.ws) = 0;
    } else if (read_status(a.ws) != 0) {
        return;
    }
    const int units = units_of(a);
    const int warp = threadIdx.x >> 5;
    if (warp == 0) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 32) {
        mbar_init(&sm.full_qk, 32 * kLoadWarps); mbar_init(&sm.full_v, 32 * kLoadWarps);
        mbar_init(&sm.qk, 1); mbar_init(&sm.qs, 1); mbar_init(&sm.pv, 1); mbar_init(&sm.ds, 1);
        mbar_init(&sm.s, 32 * kStateWarps); mbar_init(&sm.piece, 32 * kStateWarps);
        mbar_init(&sm.p, 32 * kScoreWarps); mbar_init(&sm.o, 32 * kScoreWarps);
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sm.tmem;
    if (warp < kScoreWarps) lin_scores(a, sm, units, tm);
    else if (warp < kScoreWarps + kStateWarps) lin_state(a, sm, units, tm);
    else if (warp < kScoreWarps + kStateWarps + kLoadWarps) lin_load(a, sm, units);
    else if ((threadIdx.x & 31) == 0) lin_mma(a, sm, units, tm);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tm, 512);
}

// The states the segments of a sequence start from, in place of the segments' own sums:
//   start_{i+1} = gamma^{len_i} start_i + sum_i, in the order of the job's tokens.
// One thread for 4 elements of every segment of a (sequence, head).
__global__ void __launch_bounds__(256) linattn_carry_kernel(const __grid_constant__ LinArgs a) {
    if (read_status(a.ws) != 0) return;
    const LinJob& j = a.job[blockIdx.z];
    const int i = blockIdx.x / 16, h = blockIdx.y, e = ((blockIdx.x & 15) * 256 + threadIdx.x) * 4;
    const int slots = a.table ? *a.slots_dev : a.slots;
    if (i >= slots) return;
    const Slot s = slot_of(a, i);
    if (s.seg != 0 || s.nseg == 1) return;
    const float g = a.log_decay[h];
    const size_t seq = ((size_t)s.seq * a.H + h) * D * D;
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (j.s_in) {
        if (j.s_in_t) {
            const int r = e / D, c = e % D;
            x = make_float4(j.s_in[seq + c * D + r], j.s_in[seq + (c + 1) * D + r], j.s_in[seq + (c + 2) * D + r],
                            j.s_in[seq + (c + 3) * D + r]);
        } else {
            x = *reinterpret_cast<const float4*>(j.s_in + seq + e);
        }
    }
    for (int k = 0; k < s.nseg; ++k) {
        const int at = j.rev ? i + s.nseg - 1 - k : i + k;
        float4* p = reinterpret_cast<float4*>(j.seg + ((size_t)at * a.H + h) * D * D + e);
        const float4 y = k + 1 < s.nseg ? *p : x;
        *p = x;
        const float w = expf(g * (float)slot_of(a, at).len);
        x = make_float4(w * x.x + y.x, w * x.y + y.y, w * x.z + y.z, w * x.w + y.w);
    }
}

// Packed sequences: checks the offsets (cu[0] = 0, non-decreasing, cu[N] = T_total), starts the
// status word and lists the slots, the segments of each sequence next to one another. One CTA.
__global__ void __launch_bounds__(1024)
    linattn_table_kernel(const int64_t* __restrict__ cu, int N, int64_t T_total, int64_t seg_len, int slots_max,
                         Slot* __restrict__ table, int* __restrict__ slots, uint8_t* __restrict__ ws) {
    __shared__ int bad, carry;
    __shared__ int scan[1024];
    const int tid = threadIdx.x;
    if (tid == 0) {
        bad = (cu[0] != 0 || cu[N] != T_total) ? 1 : 0;
        carry = 0;
    }
    __syncthreads();
    for (int n = tid; n < N; n += blockDim.x)
        if (cu[n + 1] < cu[n]) bad = 1;
    __syncthreads();
    if (bad) {   // nothing below is safe on such offsets
        if (tid == 0) {
            *slots = 0;
            *reinterpret_cast<int*>(ws) = KDA_ERR_OFFSETS;
        }
        return;
    }
    for (int b = 0; b < N; b += blockDim.x) {
        const int n = b + tid;
        const int64_t t0 = n < N ? cu[n] : 0, len = n < N ? cu[n + 1] - t0 : 0;
        const int cnt = n < N ? (len > 0 ? (int)((len + seg_len - 1) / seg_len) : 1) : 0;
        scan[tid] = cnt;
        __syncthreads();
        for (int o = 1; o < (int)blockDim.x; o <<= 1) {
            const int x = tid >= o ? scan[tid - o] : 0;
            __syncthreads();
            scan[tid] += x;
            __syncthreads();
        }
        const int first = carry + scan[tid] - cnt;
        for (int k = 0; k < cnt; ++k) {
            const int64_t left = len - k * seg_len;
            if (first + k < slots_max) table[first + k] = Slot{t0 + k * seg_len, (int32_t)(left < seg_len ? left : seg_len), n, k, cnt};
        }
        __syncthreads();
        if (tid == blockDim.x - 1) carry += scan[tid];
        __syncthreads();
    }
    if (tid == 0) {
        *slots = carry;
        *reinterpret_cast<int*>(ws) = 0;
    }
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
    if (sh->N * sh->H >= (int64_t(1) << 28)) return KDA_ERR_SHAPE;   // units are counted in 32 bits
    if (sh->groups < 0 || (sh->groups > 1 && sh->H % sh->groups != 0)) return KDA_ERR_SHAPE;
    return KDA_OK;
}

// How the tokens are split. A unit is a (segment, head, job); each takes its chunks one after
// another on one SM. With fewer units than SMs a sequence is cut into segments: their own state
// sums come first (state-only units, about 0.4 of a full one's time), then the states they start
// from, then all segments at once.
struct Plan {
    int64_t seg_len;   // tokens, a multiple of the chunk
    int nseg;          // segments of a fixed-length sequence (packed: of T_total tokens at most)
    int slots;         // fixed: slots; packed: most slots
};
Plan plan_of(const kda_linattn_shape* sh, bool packed, int jobs) {
    const int64_t chunks = (sh->T + LC - 1) / LC;
    // packed: as if one sequence held all tokens, which bounds the longest segment whatever the lengths
    const int64_t rows = (packed ? 1 : sh->B) * sh->H * jobs, pre = (packed ? 1 : sh->B) * sh->H * (jobs > 1 ? 2 : 1);
    int best = 1;
    double least = 0.0;
    for (int s = 1; s <= 64 && s <= (chunks > 0 ? chunks : 1); ++s) {
        const double len = (double)((chunks + s - 1) / s);
        double t = (double)((rows * s + kSMs - 1) / kSMs) * (len + kUnitChunks);
        if (s > 1) t += (double)((pre * (s - 1) + kSMs - 1) / kSMs) * (kStateOnly * len + kUnitChunks) + kSplitChunks;
        if (s == 1 || t < least) { least = t; best = s; }
    }
    Plan p;
    p.seg_len = (chunks + best - 1) / best * LC;
    if (p.seg_len < LC) p.seg_len = LC;
    p.nseg = (int)(chunks > 0 ? (sh->T + p.seg_len - 1) / p.seg_len : 1);
    p.slots = packed ? (int)(sh->N + sh->T / p.seg_len) : (int)(sh->B * p.nseg);
    return p;
}

struct LinLayout {
    size_t table, seg[2], share_q, share_k, total;
};
LinLayout layout_of(const kda_linattn_shape* sh, bool packed, bool backward) {
    const Plan p = plan_of(sh, packed, backward ? 3 : 1);
    LinLayout l;
    size_t o = 1024;   // the status word, at byte 64 the number of slots
    l.table = o; o += packed ? align_up((size_t)p.slots * sizeof(Slot), 1024) : 0;
    const size_t states = p.nseg > 1 ? (size_t)p.slots * sh->H * D * D * sizeof(float) : 0;
    l.seg[0] = o; o += states;
    l.seg[1] = o; o += backward ? states : 0;
    const size_t share = backward && groups_of(sh) > 1 ? align_up((size_t)(sh->B * sh->T * sh->H) * D * sizeof(float), 1024) : 0;
    l.share_q = o; o += share;
    l.share_k = o; o += share;
    l.total = o;
    return l;
}

kda_status common_checks(const kda_linattn_shape* sh, const int64_t* cu, const void* ws, size_t bytes, bool backward) {
    const kda_status st = check_shape(sh, cu != nullptr);
    if (st != KDA_OK) return st;
    if (!ws || bytes < layout_of(sh, cu != nullptr, backward).total) return KDA_ERR_WORKSPACE;
    if (misaligned(ws) || (reinterpret_cast<uintptr_t>(cu) & 7u)) return KDA_ERR_ALIGN;
    return KDA_OK;
}

// Launches for `jobs` sums over the shape's tokens. seg[0], seg[1]: the segment states of job 0 and,
// transposed for job 1, of job 2 (the backward's two reversed jobs sum the same state).
kda_status run_jobs(const kda_linattn_shape* sh, LinArgs& a, int jobs, const int64_t* cu, const float* log_decay, uint8_t* ws,
                    const LinLayout& lay, cudaStream_t s) {
    const Plan p = plan_of(sh, cu != nullptr, jobs);
    const cudaError_t e = cudaFuncSetAttribute(linattn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(LinSmem) + 1024);
    if (e != cudaSuccess) {
        set_last_error_text(cudaGetErrorString(e));
        return KDA_ERR_CUDA;
    }
    a.log_decay = log_decay;
    a.T = sh->T;
    a.H = (int)sh->H;
    a.ws = ws;
    a.seg_len = p.seg_len;
    a.nseg = p.nseg;
    a.slots = p.slots;
    a.jobs = jobs;
    a.first = 1;
    for (int i = 0; i < jobs; ++i) {
        a.job[i].seg = reinterpret_cast<float*>(ws + lay.seg[i > 0]);
        a.job[i].seg_t = i == 1;
    }
    if (cu) {
        Slot* const table = reinterpret_cast<Slot*>(ws + lay.table);
        int* const slots = reinterpret_cast<int*>(ws + 64);
        linattn_table_kernel<<<1, 1024, 0, s>>>(cu, (int)sh->N, sh->T, p.seg_len, p.slots, table, slots, ws);
        a.table = table;
        a.slots_dev = slots;
        a.first = 0;
    }
    auto launch = [&](const LinArgs& x) {
        const int64_t units = (int64_t)p.slots * sh->H * x.jobs;
        linattn_kernel<<<(unsigned)(units < kSMs ? units : kSMs), kLinThreads, sizeof(LinSmem) + 1024, s>>>(x);
    };
    if (p.nseg > 1) {
        LinArgs b = a;
        b.state_only = 1;
        if (jobs > 1) { b.jobs = 2; b.job[1] = a.job[2]; }
        launch(b);
        b.first = a.first = 0;
        linattn_carry_kernel<<<dim3((unsigned)p.slots * 16, (unsigned)sh->H, (unsigned)b.jobs), 256, 0, s>>>(b);
    }
    if (p.slots > 0) launch(a);
    return KDA_OK;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" size_t kda_linattn_workspace_size(const kda_linattn_shape* shape, int backward) {
    // the same shape may be used with or without offsets
    if (!shape || (check_shape(shape, true) != KDA_OK && check_shape(shape, false) != KDA_OK)) return 0;
    size_t most = 0;
    for (int packed = 0; packed < 2; ++packed)
        if (check_shape(shape, packed != 0) == KDA_OK) {
            const size_t b = layout_of(shape, packed != 0, backward != 0).total;
            if (b > most) most = b;
            // the backward's workspace serves the forward too
            const size_t f = backward ? layout_of(shape, packed != 0, false).total : 0;
            if (f > most) most = f;
        }
    return most;
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
    a.job[0] = LinJob{q, k, v, G, G, 1, o, nullptr, h0, hT, nullptr, 0, 0, 0, hT ? 3 : 2, 1.0f, shape->scale};
    const kda_status rs = run_jobs(shape, a, 1, cu_seqlens, log_decay, static_cast<uint8_t*>(workspace),
                                   layout_of(shape, cu_seqlens != nullptr, false), static_cast<cudaStream_t>(stream));
    return rs != KDA_OK ? rs : launched("kda_linattn_fwd launch");
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
    const LinLayout lay = layout_of(shape, cu_seqlens != nullptr, true);
    float* const share_q = G > 1 ? reinterpret_cast<float*>(ws + lay.share_q) : nullptr;
    float* const share_k = G > 1 ? reinterpret_cast<float*>(ws + lay.share_k) : nullptr;
    const float sc = shape->scale;
    LinArgs a{};
    // parts of the decayed keys: three (fp32-accurate) where the state itself is an output
    a.job[0] = LinJob{do_, v, k, 1, 1, G, dq, share_q, h0, nullptr, nullptr, 1, 0, 0, 2, 1.0f, sc};
    a.job[1] = LinJob{v, do_, q, 1, 1, G, dk, share_k, dhT, nullptr, nullptr, 1, 1, 1, 2, sc, 1.0f};
    a.job[2] = LinJob{k, q, do_, G, G, 1, dv, nullptr, dhT, dh0, nullptr, 0, 0, 1, dh0 ? 3 : 2, sc, 1.0f};
    const kda_status rs = run_jobs(shape, a, 3, cu_seqlens, log_decay, ws, lay, s);
    if (rs != KDA_OK) return rs;
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
