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
//
// A job goes through its tokens in chunks of 128, the rows of a tcgen05 tile: scores Q K^T, their decays, times V;
// Q S^T with the state the chunk starts from; the state's sum of decayed keys times values. That is 4 products of
// 128 x 128 x 128 with fp32 sums in tensor memory (the last of them twice or three times, see three_parts), 2600 cycles
// of the tensor core, and 128 KB in and out, about 2700 cycles of an SM's share of HBM. One CTA on an SM, by its
// shared and tensor memory, has one chunk at work and part of the next: the chain from one state to the next (decayed
// keys 1200 cycles, state 640, its bf16 copy 600, Q S^T 600, the state's sum 1060, waits between them) takes
// about 5700 cycles, and it bounds the prompts. A chunk with two parts (kFineTokens) has two products more and takes 1.4
// times as long. Measured: T = 4096, 152 heads forward 118 us, 5.2 TB/s of DRAM traffic; T = 8192, 96 heads backward 414 to 427
// us by the clocks, for 12 tensors of 201 MB (5.7 of 6.7 TB/s; 7 would do if the jobs shared their reads).
// Not faster, each against the code of its time: the jobs of a head side by side, which do share them in L2 (T = 4096,
// 152 heads: 1.03 instead of 1.41 GB read, 322 instead of 302 us); the next chunk's state sum issued before this one's
// outputs (8192 x 96 backward 409 against 382 us); a whole split call in one cooperative kernel (T = 4096, 32 heads forward 79
// against 71 us); chunks of one and of two parts as two instances of the roles' code (T = 4096, 32 heads 77 against 70 us).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>
#include <type_traits>
#include <cuda.h>
#include "kda_internal.cuh"
#include "umma_bf16.cuh"

namespace kda {
void set_last_error_text(const char* msg);

namespace {

constexpr int LC = 128;                       // tokens of a chunk
constexpr int kSMs = 152;                     // of a GB300; one persistent CTA on each
// the cost model of the split, in chunk times of a full unit (2.7 us): a state-only chunk, the start of a unit, the two more
// launches, and each state that is carried (fitted to T = 512 .. 16384 with 1 .. 64 heads cut into 1 .. 64 segments)
constexpr double kStateOnly = 0.55, kUnitChunks = 1.0, kSplitChunks = 4.5, kCarried = 1.0 / 40;
// The chunks that start within so many tokens of where a sequence starts, in the job's direction, have their scores, and
// the state that they read, in two bf16 parts (16 significant bits). Rounded once, these put an output off by 1.4 times
// its own rounding in the mean square where many scores make up a row, but by up to 2.5 times where a single one does, as
// in the first rows. It goes by a row's place in its sequence alone, so that a sequence has the same precision
// whatever shares its call. (By the call's tokens, short calls in two parts and others in one: T = 8192, 96 heads backward 396
// us, packed six with 96 heads forward 187; by place 417 and 215; two parts throughout 556 and 244, and as much with
// two parts for heads that decay by e^-0.5 a token too, whose rows are few scores everywhere: they hold up the rest.)
constexpr int kFineTokens = 512;
constexpr uint32_t kTile = LC * D * 2;        // a bf16 operand tile [128][128], two 64-column panels

// One sum over tokens in the roles' names. Row i of a chunk of L rows, with the state S the
// chunk starts from (e = 1 forward, 0 reversed: a token's decay applies before or after its read):
//   out_i = scale (sum_{j <= i} gamma^{i-j} (q_i . k_j) v_j + gamma^{i+e} S q_i)
//   S    <- gamma^L S + sum_j gamma^{L-e-j} v_j k_j^T
// The adjoint state of a reversed job is scale times its S: s_in is divided and s_out multiplied by it.
struct LinJob {
    int q, k, v;                 // which of LinArgs' tensors
    uint16_t* out;               // [tokens, H, 128] bf16, or
    float* share;                // [tokens, H, 128] fp32: each value head's share of a grouped sum
    const float* s_in;           // initial state [N, H, 128, 128], may be NULL
    float* s_out;                // final state, may be NULL
    float* seg;                  // states of the segments [slots, H, 128, 128]
    int s_in_t, seg_t;           // s_in, seg are stored transposed
    int rev;                     // tokens from last to first
    int exact;                   // the state is an output: fp32-accurate (else as good as its bf16 copy needs)
    float s_scale;               // of s_in and s_out over S: 1, or scale
};

// A slot is a segment of a sequence; a sequence has one at least, an empty one too.
struct Slot {
    int64_t t0;         // first token
    int32_t len, seq;
    int32_t seg, nseg;  // its place among the sequence's segments,
    int32_t before, after;   // and the sequence's tokens on either side of it
};

struct LinArgs {
    CUtensorMap map[4];          // [tokens, H / group, 128] bf16 in boxes of 128 tokens x 64 channels
    CUtensorMap out_map[3];      // each job's out or share in boxes of 32 tokens x 128 bytes
    int group[4];                // value heads that share a head of each
    LinJob job[3];
    int jobs;
    int state_only;              // the segments' own states to seg, nothing else
    int first;                   // the first kernel of the call on this workspace: clears its status word
    Slot* table;                 // packed: slots and their number, written by linattn_table_kernel, or
    const int* slots_dev;
    const int64_t* cu;           // the offsets of few whole sequences, from which each block writes the slot of its unit
    int slots;                   // fixed length: nseg segments of seg_len tokens per sequence; with cu: N
    int nseg;
    int64_t seg_len, T;
    const float* log_decay;
    float scale;
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
    s.before = (int32_t)at;
    s.after = (int32_t)(left - s.len);
    return s;
}

// Held by value: the kernel's loops store to shared memory, and a pointer into the parameters would
// be read again after every store.
struct Unit {
    int64_t t0;
    int len, h, rev;
    int job, q, k, v;              // tensors
    uint8_t* out;                  // out or share
    bool fp32;
    float scale, g;                // g: log decay
    float in_scale, out_scale;     // what the state is multiplied with on its way in and out
    int exact, after, done;        // tokens of the sequence, in the unit's order, still to come after it and before it
    const float* s_in;             // where this unit's state comes from and goes to, NULL: zero, not wanted
    float* s_out;
    int s_in_t;
};
__device__ __forceinline__ Unit unit_of(const LinArgs& a, int u) {
    const int per = a.jobs * a.H;
    const int i = u / per, r = u - i * per, ji = r / a.H;
    const Slot s = slot_of(a, i);
    const LinJob j = a.job[ji];
    Unit x;
    x.h = r - ji * a.H;
    x.t0 = s.t0;
    x.len = s.len;
    x.rev = j.rev;
    x.q = j.q; x.k = j.k; x.v = j.v;
    x.job = ji;
    x.fp32 = j.share != nullptr;
    x.out = x.fp32 ? reinterpret_cast<uint8_t*>(j.share) : reinterpret_cast<uint8_t*>(j.out);
    x.scale = a.scale;
    x.in_scale = x.out_scale = 1.0f;
    x.g = a.log_decay[x.h];
    x.exact = j.exact;
    x.after = j.rev ? s.before : s.after;
    x.done = j.rev ? s.after : s.before;
    const size_t seq_state = ((size_t)s.seq * a.H + x.h) * D * D, seg_state = ((size_t)i * a.H + x.h) * D * D;
    const bool head = j.rev ? s.seg == s.nseg - 1 : s.seg == 0, tail = j.rev ? s.seg == 0 : s.seg == s.nseg - 1;
    if (a.state_only) {            // every segment but the last of its sequence starts from zero and leaves its sum
        x.s_in = nullptr;
        x.s_in_t = 0;
        x.s_out = tail ? nullptr : j.seg + seg_state;
        if (tail) x.len = 0;
    } else {
        // the first segment of several reads its copy too: a final state that takes the initial one's place may be there already
        const bool given = head && (s.nseg == 1 || !j.s_in);
        x.s_in = given ? (j.s_in ? j.s_in + seq_state : nullptr) : j.seg + seg_state;
        x.s_in_t = given ? j.s_in_t : j.seg_t;
        if (x.len > 0) {           // an empty sequence's state passes through unchanged
            if (given) x.in_scale = 1.0f / j.s_scale;
            x.out_scale = j.s_scale;
        }
        x.s_out = tail && j.s_out ? j.s_out + seq_state : nullptr;
    }
    return x;
}
__device__ __forceinline__ int units_of(const LinArgs& a) { return (a.slots_dev ? *a.slots_dev : a.slots) * a.H * a.jobs; }
// the units of a CTA: every round of gridDim.x units in turn from the other end, so that with slots in
// order of falling length no CTA gets the longer one each time
__device__ __forceinline__ int unit_at(int round) {
    return round * (int)gridDim.x + (int)((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// Chunk c of a unit: rows are tokens t .. t + 127 in either direction, a reversed unit's chunks are
// counted from its end; rows lo <= r < hi belong to the unit (fewer than 128 in its last chunk).
struct Chunk {
    int64_t t;
    int lo, hi;
};
__device__ __forceinline__ Chunk chunk_of(const Unit& u, int c) {
    const int left = u.len - c * LC;
    Chunk x;
    x.t = u.rev ? u.t0 + left - LC : u.t0 + (int64_t)c * LC;
    x.lo = u.rev ? max(LC - left, 0) : 0;
    x.hi = u.rev ? LC : min(left, LC);
    return x;
}
// The decayed keys of a chunk go into the state's sum as two bf16 parts (16 significant bits, 2.2e-6 of
// their size in the mean square), or as three (24) where the state is an output and the tokens still to
// come will not have decayed this chunk's share, and its error with it, by another e^-1: an output state
// is within 1e-6 of its size. (Without any decay one part is exact.) Forward with states, six sequences of 8192
// tokens in all with 96 heads: 289 us with three parts always, 215 by this rule, 197 with two always.
__device__ __forceinline__ bool three_parts(const Unit& u, int c) {
    const int left = u.after + max(u.len - (c + 1) * LC, 0);
    return u.exact && u.g != 0.0f && (left == 0 || u.g * (float)left > -1.0f);
}
__device__ __forceinline__ bool in_two_parts(const Unit& u, int c) { return u.done + c * LC < kFineTokens; }
__device__ __forceinline__ int chunks_of(const Unit& u) { return (u.len + LC - 1) / LC; }

struct LinSmem {
    // operand tiles (bf16 panels, 1024-byte aligned), K and V by chunk parity
    uint8_t K[2][kTile], V[2][kTile], Q[kTile];
    uint8_t S[kTile];        // the state the chunk starts from, [c][v], rounded to bf16
    uint8_t stage[kTile];    // output rows on their way out; before them, in two parts, the low part of S
    float diag[4][64];       // per score warp: decays inside the diagonal's 32 x 32 block
    float decay[LC];         // of the keys of a whole chunk
    // full: operands in shared memory; qk, qs, ds, pv: MMA groups done, all: of the chunk; s, p, piece, low, o:
    // operands written (state, scores, decayed keys and their low parts, decayed Q S^T); r: outputs read. Each
    // completes one phase per chunk (full_k, full_v, all: one of the two; low: per chunk with three parts).
    // A wait names a phase by its parity, so no waiter may be a whole phase behind or ahead: every wait
    // comes before an arrival of the same thread on which the barrier's next phase depends, and after
    // something that depends on the phase before. A thread that arrives twice on a barrier waits in between
    // for something that depends on all the first arrivals.
    uint64_t full_k[2], full_q, full_v[2], all[2], qk, qs, ds, pv, s, p, piece, low, o, r, end;
    uint32_t tmem;
};

// Warps 0-3: scores and outputs (thread = row of the chunk = TMEM lane). Warps 4-11: the state and the
// decayed keys (thread = half a TMEM lane's columns). Warp 12: loads. Warp 13: MMAs. Warps 14, 15 complete a warpgroup,
// the unit in which registers are handed over: 128 a thread at launch, 128 + 152 + 152 + 80 = 4 x 128.
constexpr int kScoreWarps = 4, kMainWarps = 8;
constexpr int kLinThreads = 512;
constexpr int kMainRegs = 152, kIssueRegs = 80;

// the same value in every lane of the warp, and known to be (uniform registers)
template <typename X> __device__ __forceinline__ X uniform(X x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ bool wait_warp(uint64_t* bar, int n) {
    return __all_sync(0xffffffffu, mbar_wait_asleep(bar, (uint32_t)(n & 1)));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ float low_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(f32x2 a) {
    const float2 x = parts(a);
    return pack_bf16(x.x, x.y);
}

// what bf16 leaves of a pair, itself in bf16
__device__ __forceinline__ uint32_t low_part(f32x2 p, uint32_t high) {
    return pack_bf16(fma2(two(-1.0f, -1.0f), two(low_bf16(high), high_bf16(high)), p));
}

// The chunks of a CTA's units, one after another.
struct At {
    int round, c, chunks;
    bool more;
    Unit u;
    __device__ __forceinline__ void settle(const LinArgs& a, int units) {   // the first unit from here on that has chunks
        for (c = 0;; ++round) {
            const int i = unit_at(round);
            if (!(more = i < units)) return;
            u = unit_of(a, i);
            if ((chunks = chunks_of(u)) > 0) return;
        }
    }
    __device__ __forceinline__ void first(const LinArgs& a, int units) {
        round = 0;
        settle(a, units);
    }
    __device__ __forceinline__ void next(const LinArgs& a, int units) {
        if (++c == chunks) {
            ++round;
            settle(a, units);
        }
    }
};

// --- loads, one thread
__device__ __forceinline__ void lin_load(const LinArgs& a, LinSmem& sm, int units) {
    const bool state_only = a.state_only != 0;
    struct Place { int q, k, v, h, t; };
    auto place = [](const At& x) { return Place{x.u.q, x.u.k, x.u.v, x.u.h, (int)chunk_of(x.u, x.c).t}; };
    auto tile = [&](uint8_t* dst, int which, const Place& x, uint64_t* bar) {
        const int head = x.h / a.group[which];
        mbar_arrive_expect_tx(bar, kTile);
        tma_load_3d(dst, &a.map[which], 0, head, x.t, bar);
        tma_load_3d(dst + kTile / 2, &a.map[which], 64, head, x.t, bar);
    };
    auto q_tile = [&](const Place& x) {
        if (state_only) mbar_arrive(&sm.full_q);
        else tile(sm.Q, x.q, x, &sm.full_q);
    };
    auto ahead = [&](int which, const Place& x) {
        const int head = x.h / a.group[which];
        tma_prefetch_3d(&a.map[which], 0, head, x.t);
        tma_prefetch_3d(&a.map[which], 64, head, x.t);
    };
    At x;
    x.first(a, units);
    if (!x.more) return;
    Place next = place(x);
    tile(sm.K[0], next.k, next, &sm.full_k[0]);
    tile(sm.V[0], next.v, next, &sm.full_v[0]);
    q_tile(next);
    for (int n = 0;; ++n) {
        x.next(a, units);
        if (!x.more) return;
        next = place(x);   // chunk n + 1: its keys and values once chunk n - 1 is done
        if (n > 0 && !mbar_wait(&sm.all[(n - 1) & 1], (uint32_t)(((n - 1) >> 1) & 1))) break;
        tile(sm.K[(n + 1) & 1], next.k, next, &sm.full_k[(n + 1) & 1]);
        tile(sm.V[(n + 1) & 1], next.v, next, &sm.full_v[(n + 1) & 1]);
        if (!state_only) ahead(next.q, next);   // on their way into L2: from there they arrive in time
        if (!mbar_wait(&sm.qs, (uint32_t)(n & 1))) break;
        q_tile(next);
    }
    raise_status(a.ws, KDA_ERR_TIMEOUT);
}

// --- MMAs, one thread. TMEM: scores and, in the first half of each block of 32 columns, its bf16 copy (two to a
// column), in the second half the copy's low part or, after that, the decayed keys' low parts; outputs; state sum
// [c][v]; decayed keys [c][tokens], high and middle parts (two to a column)
constexpr uint32_t kColP = 0, kColLow = 16, kColO = 128, kColDS = 256, kColHi = 384, kColMid = 448;
// A product over K = 128: eight MMAs, unrolled, descriptors a constant apart. (The thread that issues them is
// what limits it otherwise: with descriptors built one by one an MMA of 128 x 128 x 16 took 130 to 190 cycles,
// so it takes 65, the time to read its operands from shared memory.)
__device__ __forceinline__ uint64_t k_step(uint64_t d, int s) { return d + (uint64_t)((s >> 2) * (kTile / 2 / 16) + (s & 3) * 2); }
__device__ __forceinline__ uint64_t mn_step(uint64_t d, int s) { return d + (uint64_t)(s * 128); }
template <bool kBmn>
__device__ __forceinline__ void product_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add = false) {
#pragma unroll
    for (int s = 0; s < 8; ++s) umma_bf16(d, k_step(a, s), kBmn ? mn_step(b, s) : k_step(b, s), idesc, add || s > 0);
}
// A in tensor memory, `add` to what the accumulator holds; kBlocks: in the halves of blocks, else in 64 columns one after another
template <bool kBlocks>
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
#pragma unroll
    for (int s = 0; s < 8; ++s) umma_bf16_ta(d, a + 8 * s + (kBlocks ? 16 * (s >> 1) : 0), mn_step(b, s), idesc, add || s > 0);
}
__device__ __forceinline__ void lin_mma(const LinArgs& a, LinSmem& sm, int units, uint32_t tm) {
    const bool state_only = a.state_only != 0;
    constexpr uint32_t kk = idesc_bf16(128, 128, 0, 0), kn = idesc_bf16(128, 128, 0, 1);
    const uint64_t dk0 = desc_kmajor(smem_u32(sm.K[0]), LC, 0), ds = desc_mnmajor_bf16(smem_u32(sm.S), LC, 0);
    const uint64_t q = desc_kmajor(smem_u32(sm.Q), LC, 0), dv0 = desc_mnmajor_bf16(smem_u32(sm.V[0]), LC, 0);
    bool ok = true;
    int n = 0, lows = 0;
    At x;
    x.first(a, units);
    auto score = [&](int m) {   // scores of chunk m
        if (!mbar_wait(&sm.full_k[m & 1], (uint32_t)((m >> 1) & 1)) || !mbar_wait(&sm.full_q, (uint32_t)(m & 1))) return false;
        if (!state_only) product_ss<false>(tm + kColP, q, dk0 + (uint64_t)((m & 1) * (kTile / 16)), kk);
        umma_commit(&sm.qk);
        return true;
    };
    if (x.more) ok = score(0);
    for (; ok && x.more; ++n) {
        const uint32_t ph = (uint32_t)(n & 1);
        const uint64_t v = dv0 + (uint64_t)(ph * (kTile / 16));
        const bool carried = x.c > 0 || x.u.s_in, sum = x.c + 1 < x.chunks || x.u.s_out, three = sum && three_parts(x.u, x.c);
        const bool fine = in_two_parts(x.u, x.c);
        if (!(ok = mbar_wait(&sm.s, ph) && (n == 0 || mbar_wait(&sm.r, ph ^ 1u)))) break;
        tc_fence_after();
        if (!state_only && carried) {
            if (fine) product_ss<true>(tm + kColO, q, ds + (uint64_t)(kTile / 16), kn);   // its low part, in the stage
            product_ss<true>(tm + kColO, q, ds, kn, fine);
        }
        umma_commit(&sm.qs);
        if (!(ok = mbar_wait(&sm.piece, ph) && mbar_wait(&sm.full_v[n & 1], (uint32_t)((n >> 1) & 1)))) break;
        tc_fence_after();
        if (sum) {   // small parts first: the accumulator is rounded at its size
            product_ts<false>(tm + kColDS, tm + kColMid, v, kn, false);
            product_ts<false>(tm + kColDS, tm + kColHi, v, kn, true);
        }
        if (!three) umma_commit(&sm.ds);
        if (!(ok = mbar_wait(&sm.o, ph) && mbar_wait(&sm.p, ph))) break;
        tc_fence_after();
        if (!state_only) {
            if (fine) product_ts<true>(tm + kColO, tm + kColP + kColLow, v, kn, carried);
            product_ts<true>(tm + kColO, tm + kColP, v, kn, carried || fine);
        }
        umma_commit(&sm.pv);
        if (three) {
            if (!(ok = mbar_wait(&sm.low, (uint32_t)(lows++ & 1)))) break;
            tc_fence_after();
            product_ts<true>(tm + kColDS, tm + kColP + kColLow, v, kn, true);
            umma_commit(&sm.ds);
        }
        umma_commit(&sm.all[n & 1]);
        x.next(a, units);
        // the next chunk's scores now: they and their decays need no state
        if (x.more) ok = score(n + 1);
    }
    if (!ok) raise_status(a.ws, KDA_ERR_TIMEOUT);
    umma_commit(&sm.end);   // no MMA is in flight when the tensor memory is freed
    mbar_wait(&sm.end, 0);
}

// --- scores -> decayed bf16 scores in TMEM; outputs -> shared memory -> global, a warp's 32 rows by TMA (or,
// in a chunk with rows of a neighbour, row by row)
__device__ __forceinline__ void lin_scores(const LinArgs& a, LinSmem& sm, int units, uint32_t tm) {
    const bool state_only = a.state_only != 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t lanes = tm + ((uint32_t)(32 * warp) << 16);
    float* const diag = sm.diag[warp];
    uint8_t* const stage = sm.stage + warp * 4096;   // rows 32 warp .. of the tile
    const int heads = a.H;
    bool ok = true;
    int n = 0;
    for (int round = 0; ok; ++round) {
        const int at = unit_at(round);
        if (at >= units) break;
        const Unit u = unit_of(a, at);
        const int chunks = chunks_of(u);
        if (chunks == 0) continue;
        const float g = u.g;
        const bool rev = u.rev != 0;
        // scale gamma^{|row - col|}, row = 32 warp + lane, col = 32 b + x. Off the diagonal's
        // block it is gamma^{32 |warp - b| - 31} f[x], f[x] = scale gamma^{31 + lane - x} (reversed:
        // 31 - lane + x): no exponent is negative. On it, diag[lane - x + 31].
        const float scale = u.scale;
        f32x2 f[16];
#pragma unroll
        for (int x = 0; x < 16; ++x)
            f[x] = two(scale * decay_pow(g, 31 + (rev ? 2 * x - lane : lane - 2 * x)),
                       scale * decay_pow(g, 31 + (rev ? 2 * x + 1 - lane : lane - 2 * x - 1)));
        __syncwarp();
        diag[31 + lane] = diag[31 - lane] = scale * decay_pow(g, lane);
        __syncwarp();
        const uint32_t keep = rev ? 0xffffffffu << lane : 0xffffffffu >> (31 - lane);   // columns that count in its block
        const float far1 = decay_pow(g, 1), far2 = decay_pow(g, 33), far3 = decay_pow(g, 65);
        // from the far end to the diagonal's block, so that its table is read when Q S^T, which leaves
        // shared memory no read cycles, is over; zeros beyond it
        auto copy = [&](auto in_parts) {
            constexpr bool kFine = decltype(in_parts)::value;
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                const int b = rev ? 3 - i : i, away = rev ? b - warp : warp - b;
                uint32_t w[16], low[16];
                if (away < 0) {
#pragma unroll
                    for (int x = 0; x < 16; ++x) w[x] = low[x] = 0u;
                } else {
                    uint32_t r[32];
                    tmem_ld32_issue(lanes + kColP + 32 * b, r);
                    if (away > 0) {
                        const float base = away == 1 ? far1 : away == 2 ? far2 : far3;
                        const f32x2 base2 = two(base, base);
                        tmem_wait_ld(r);
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            const f32x2 p = mul2(two(r[2 * x], r[2 * x + 1]), mul2(base2, f[x]));
                            w[x] = pack_bf16(p);
                            if (kFine) low[x] = low_part(p, w[x]);
                        }
                    } else {
                        const float* const d = diag + 31 + lane;
                        tmem_wait_ld(r);
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            const float p0 = __uint_as_float(r[2 * x]) * d[-2 * x], p1 = __uint_as_float(r[2 * x + 1]) * d[-2 * x - 1];
                            const f32x2 p = two((keep >> (2 * x)) & 1u ? p0 : 0.0f, (keep >> (2 * x + 1)) & 1u ? p1 : 0.0f);
                            w[x] = pack_bf16(p);
                            if (kFine) low[x] = low_part(p, w[x]);
                        }
                    }
                }
                tmem_st16_issue(lanes + kColP + 32 * b, w);   // columns that have been read
                if (kFine) tmem_st16_issue(lanes + kColP + 32 * b + kColLow, low);
            }
        };
        for (int c = 0; c < chunks; ++c, ++n) {
            if (!(ok = wait_warp(&sm.qk, n))) break;
            tc_fence_after();
            const bool fine = in_two_parts(u, c);
            if (!state_only) {
                if (fine) copy(std::true_type{});
                else copy(std::false_type{});
                tmem_wait_st_all();
            }
            tc_fence_before();
            mbar_arrive(&sm.p);
            if (!(ok = wait_warp(&sm.pv, n))) break;
            tc_fence_after();
            if (state_only) {
                mbar_arrive(&sm.r);
                continue;
            }
            const Chunk k = chunk_of(u, c);
            const int r0 = 32 * warp;
            // the outputs' columns are free once read, the stage, where the next chunk may want it for the low part of
            // its state, once it has been sent
            const bool late = fine || c + 1 == chunks;
            const bool all = r0 >= k.lo && r0 + 32 <= k.hi;
            // a tile of 32 rows x 128 bytes at a time, 32 or 64 columns; two are staged at once
            auto send = [&](int tile, int slot) {
                uint8_t* const from = stage + slot * (kTile / 2);
                if (all) {
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_3d(from, &a.out_map[u.job], tile * (u.fp32 ? 32 : 64), u.h, (int)k.t + r0);
                        bulk_commit();
                    }
                } else {
                    __syncwarp();
                    const int64_t pitch = (int64_t)heads * D * (u.fp32 ? 4 : 2);
#pragma unroll 1
                    for (int i = lane >> 3; i < 32; i += 4)
                        if (r0 + i >= k.lo && r0 + i < k.hi)
                            *reinterpret_cast<uint4*>(u.out + (k.t + r0 + i) * pitch + (int64_t)u.h * D * (u.fp32 ? 4 : 2) + tile * 128 +
                                                      (lane & 7) * 16) =
                                *reinterpret_cast<const uint4*>(from + panel_off_bf16(i, lane & 7, LC));
                }
            };
            auto staged = [&] {   // what was staged before has been read
                if (lane == 0) bulk_wait_read_all();
                __syncwarp();
            };
            staged();
            if (!u.fp32) {
#pragma unroll 1
                for (int t = 0; t < 2; ++t) {
                    uint32_t x[32], y[32];
                    tmem_ld32_issue(lanes + kColO + 64 * t, x);
                    tmem_ld32_issue(lanes + kColO + 64 * t + 32, y);
                    tmem_wait_ld(x);
                    tmem_after_wait(y);
                    if (t == 1) {
                        tc_fence_before();
                        if (!late) mbar_arrive(&sm.r);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        *reinterpret_cast<uint4*>(stage + t * (kTile / 2) + panel_off_bf16(lane, i, LC)) =
                            make_uint4(pack_bf16(two(x[8 * i], x[8 * i + 1])), pack_bf16(two(x[8 * i + 2], x[8 * i + 3])),
                                       pack_bf16(two(x[8 * i + 4], x[8 * i + 5])), pack_bf16(two(x[8 * i + 6], x[8 * i + 7])));
                        *reinterpret_cast<uint4*>(stage + t * (kTile / 2) + panel_off_bf16(lane, 4 + i, LC)) =
                            make_uint4(pack_bf16(two(y[8 * i], y[8 * i + 1])), pack_bf16(two(y[8 * i + 2], y[8 * i + 3])),
                                       pack_bf16(two(y[8 * i + 4], y[8 * i + 5])), pack_bf16(two(y[8 * i + 6], y[8 * i + 7])));
                    }
                    send(t, t);
                }
            } else {
#pragma unroll 1
                for (int t = 0; t < 4; ++t) {
                    if (t == 2) staged();
                    uint32_t x[32];
                    tmem_ld32_issue(lanes + kColO + 32 * t, x);
                    tmem_wait_ld(x);
                    if (t == 3) {
                        tc_fence_before();
                        if (!late) mbar_arrive(&sm.r);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4*>(stage + (t & 1) * (kTile / 2) + panel_off_bf16(lane, i, LC)) =
                            make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                    send(t, t & 1);
                }
            }
            if (late) {
                staged();
                mbar_arrive(&sm.r);
            }
        }
    }
    if (lane == 0) bulk_wait_all();
    if (!ok && lane == 0) raise_status(a.ws, KDA_ERR_TIMEOUT);
}

// --- state in registers and its bf16 copy for the next chunk; decayed keys as bf16 parts; Q S^T decayed by row
__device__ __forceinline__ void lin_main(const LinArgs& a, LinSmem& sm, int units, uint32_t tm) {
    const bool state_only = a.state_only != 0;
    const int warp = uniform((int)((threadIdx.x >> 5) & 3)), lane = threadIdx.x & 31, half = uniform((int)((threadIdx.x - 32 * kScoreWarps) >> 7));
    const int row = 32 * warp + lane;              // TMEM lane: output row, or key channel of the state
    const uint32_t lanes = tm + ((uint32_t)(32 * warp) << 16), wide = lanes + 64 * half;
    // decayed keys: this warp's channels 32 warp + .., tokens 64 half + ..; ldmatrix row of this thread
    const int jl = 64 * half + 8 * (lane >> 4) + (lane & 7), cl = 4 * warp + ((lane >> 3) & 1);
    const int jr = 64 * half + 2 * (lane & 3);     // first token of its fragment register 0
    const uint32_t key0 = smem_u32(sm.K[0]);
    bool ok = true;
    int n = 0;
    f32x2 s[32];                                   // S[v][row], v = 64 half + ..
    for (int round = 0; ok; ++round) {
        const int at = unit_at(round);
        if (at >= units) break;
        const Unit u = unit_of(a, at);
        const int chunks = chunks_of(u);
        if (u.s_in && u.s_in_t) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const float4 x = *reinterpret_cast<const float4*>(u.s_in + row * D + 64 * half + 2 * i);
                s[i] = two(u.in_scale * x.x, u.in_scale * x.y); s[i + 1] = two(u.in_scale * x.z, u.in_scale * x.w);
            }
        } else if (u.s_in) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                s[i] = two(u.in_scale * u.s_in[(64 * half + 2 * i) * D + row], u.in_scale * u.s_in[(64 * half + 2 * i + 1) * D + row]);
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) s[i] = 0ull;
        }
        const float w_state = u.scale * decay_pow(u.g, u.rev ? LC - 1 - row : row + 1);
        const f32x2 w2 = two(w_state, w_state);
        const float whole_decay = decay_pow(u.g, LC);
        // the decays of the tokens of a whole chunk in fp32 (every warp writes the same values), and those of tokens
        // jr + 8 i and the next as w = w1 + w2 in bf16. Only for a unit with chunks: the last state sum of the one
        // before has been waited for, which every warp's last read of its decays comes before. A unit without chunks
        // has nothing to wait for: its decays, written by a warp that is behind, would replace the next unit's.
        uint32_t wk1[8], wk2[8];
        if (chunks > 0) {
#pragma unroll
            for (int i = 0; i < LC; i += 32) sm.decay[lane + i] = decay_pow(u.g, u.rev ? lane + i + 1 : LC - 1 - (lane + i));
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int j = jr + 8 * i;
                const float x = sm.decay[j], y = sm.decay[j + 1];
                wk1[i] = pack_bf16(x, y);
                wk2[i] = pack_bf16(x - low_bf16(wk1[i]), y - high_bf16(wk1[i]));
            }
        }
        for (int c = 0; ok && chunks > 0; ++c) {
            if (c > 0) {   // the state sum of chunk c - 1 is there, its decayed keys are no longer needed
                if (!(ok = wait_warp(&sm.ds, n - 1))) break;
                tc_fence_after();
            }
            const bool carried = c > 0 || u.s_in, sum = c + 1 < chunks || (c < chunks && u.s_out), three = sum && three_parts(u, c);
            const bool fine = in_two_parts(u, c);
            // 32 tokens x 16 channels of K, the g-th of this warp's four blocks
            auto fragments = [&](int g, uint32_t (&x)[8]) {
                const int j = jl + 32 * (g >> 1), cc = cl + 2 * (g & 1);
                ldmatrix4_trans(key0 + (uint32_t)(n & 1) * kTile + panel_off_bf16(j, cc, LC), x[0], x[1], x[2], x[3]);
                ldmatrix4_trans(key0 + (uint32_t)(n & 1) * kTile + panel_off_bf16(j + 16, cc, LC), x[4], x[5], x[6], x[7]);
            };
            auto place = [&](int g) { return lanes + ((uint32_t)(16 * (g & 1)) << 16) + 32 * half + 16 * (g >> 1); };
            auto low_place = [&](int g) { return lanes + ((uint32_t)(16 * (g & 1)) << 16) + kColP + 64 * half + 32 * (g >> 1) + kColLow; };
            // where a thread's low parts of block g wait: the block's own bytes of K, which nothing else reads
            // once it is in fragments and the scores are done
            auto wait_place = [&](int g, int e) {
                return sm.K[n & 1] + panel_off_bf16(64 * half + 32 * (g >> 1) + lane, 4 * warp + 2 * (g & 1) + e, LC);
            };
            if (c < chunks) {
                // decayed keys, transposed to [channel][token], to tensor memory: first, while the scores and
                // outputs of chunk c - 1 leave shared memory read cycles
                if (!(ok = wait_warp(&sm.full_k[n & 1], n >> 1))) break;
                const Chunk k = chunk_of(u, c);
                const bool whole = k.hi - k.lo == LC;
                if (!whole) {   // rows of a neighbour in V: their scores are zero, and zero times an infinity is not
                    if (!(ok = __all_sync(0xffffffffu, mbar_wait_asleep(&sm.full_v[n & 1], (uint32_t)((n >> 1) & 1))))) break;
                    if (row < k.lo || row >= k.hi)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<uint4*>(sm.V[n & 1] + panel_off_bf16(row, 8 * half + i, LC)) = make_uint4(0u, 0u, 0u, 0u);
                    fence_async_smem();
                }
                if (sum && whole && !three) {
                    // w1 x = hi + e without error (the error of a rounded product has 8 bits), mid = w2 x + e
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        uint32_t x[8], hi[8], mi[8];
                        fragments(g, x);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int w = 4 * (g >> 1) + (i >> 1);
                            const __nv_bfloat162 y = *reinterpret_cast<const __nv_bfloat162*>(&x[i]);
                            const __nv_bfloat162 w1 = *reinterpret_cast<const __nv_bfloat162*>(&wk1[w]);
                            const __nv_bfloat162 h = __hmul2_rn(w1, y);
                            const __nv_bfloat162 m = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&wk2[w]), y, __hfma2(w1, y, __hneg2(h)));
                            hi[i] = *reinterpret_cast<const uint32_t*>(&h);
                            mi[i] = *reinterpret_cast<const uint32_t*>(&m);
                        }
                        tmem_st_frag_issue(place(g) + kColMid, mi);
                        tmem_st_frag_issue(place(g) + kColHi, hi);
                    }
                } else if (sum) {   // three parts, or rows of a neighbour among the tokens: in fp32
                    if (three && !(ok = wait_warp(&sm.qk, n))) break;
#pragma unroll 1
                    for (int g = 0; g < 4; ++g) {
                        uint32_t x[8], hi[8], mi[8], lo[8];
                        fragments(g, x);
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            const int t = jr + 32 * (g >> 1) + 8 * m;
                            const bool mine0 = t >= k.lo && t < k.hi, mine1 = t + 1 >= k.lo && t + 1 < k.hi;
                            // gamma^{L-1-t} (reversed, counted from the end: gamma^{t+1-lo}) is at t + 128 - L (t - lo)
                            const int e = u.rev ? t - k.lo : t + LC - k.hi;
                            const f32x2 w = two(sm.decay[mine0 ? e : 0], sm.decay[mine1 ? e + 1 : 0]);
                            const uint32_t mask = (mine0 ? 0xffffu : 0u) | (mine1 ? 0xffff0000u : 0u);
                            const f32x2 minus = two(-1.0f, -1.0f);
#pragma unroll
                            for (int i = 2 * m; i < 2 * m + 2; ++i) {
                                x[i] &= mask;
                                f32x2 p = mul2(w, two(low_bf16(x[i]), high_bf16(x[i])));
                                hi[i] = pack_bf16(p);
                                p = fma2(minus, two(low_bf16(hi[i]), high_bf16(hi[i])), p);
                                mi[i] = pack_bf16(p);
                                p = fma2(minus, two(low_bf16(mi[i]), high_bf16(mi[i])), p);
                                lo[i] = pack_bf16(p);
                            }
                        }
                        tmem_st_frag_issue(place(g) + kColMid, mi);
                        tmem_st_frag_issue(place(g) + kColHi, hi);
                        if (three) {
                            *reinterpret_cast<uint4*>(wait_place(g, 0)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                            *reinterpret_cast<uint4*>(wait_place(g, 1)) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
                        }
                    }
                }
                tmem_wait_st_all();
                tc_fence_before();
                mbar_arrive(&sm.piece);
            }
            if (c > 0 && (c < chunks || u.s_out)) {   // the state after chunk c - 1
                const float w = c < chunks ? whole_decay : decay_pow(u.g, u.len - (c - 1) * LC);
                const f32x2 decay = two(w, w);
                uint32_t r[2][32];
                tmem_ld32_issue(wide + kColDS, r[0]);
                tmem_ld32_issue(wide + kColDS + 32, r[1]);
                tmem_wait_ld(r[0]);
                tmem_after_wait(r[1]);
#pragma unroll
                for (int i = 0; i < 32; ++i) s[i] = fma2(decay, s[i], two(r[i >> 4][2 * (i & 15)], r[i >> 4][2 * (i & 15) + 1]));
            }
            if (c == chunks) break;
            if (!state_only && carried) {   // sm.S was last read before the state sum just waited for
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint4*>(sm.S + panel_off_bf16(row, 8 * half + i, LC)) =
                        make_uint4(pack_bf16(s[4 * i]), pack_bf16(s[4 * i + 1]), pack_bf16(s[4 * i + 2]), pack_bf16(s[4 * i + 3]));
                if (fine) {   // its low part where the outputs are staged later
                    if (n > 0 && !(ok = wait_warp(&sm.r, n - 1))) break;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] = low_part(s[4 * i + e], pack_bf16(s[4 * i + e]));
                        *reinterpret_cast<uint4*>(sm.stage + panel_off_bf16(row, 8 * half + i, LC)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                fence_async_smem();
            }
            tc_fence_before();
            mbar_arrive(&sm.s);
            // scale gamma^{..} Q S^T, the rows' decays, before the scores' part is added to it
            if (!(ok = wait_warp(&sm.qs, n))) break;
            if (!state_only && carried) {
                tc_fence_after();
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    uint32_t x[32];
                    tmem_ld32_issue(wide + kColO + 32 * b, x);
                    tmem_wait_ld(x);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float2 z = parts(mul2(w2, two(x[i], x[i + 1])));
                        x[i] = __float_as_uint(z.x);
                        x[i + 1] = __float_as_uint(z.y);
                    }
                    tmem_st32_issue(wide + kColO + 32 * b, x);
                }
                tmem_wait_st_all();
                tc_fence_before();
            }
            mbar_arrive(&sm.o);
            if (three) {   // the low parts: beside the scores' bf16 copy, once that is made
                if (!(ok = wait_warp(fine ? &sm.pv : &sm.p, n))) break;   // (qs: pv of the chunk before is over)
                tc_fence_after();
#pragma unroll 1
                for (int g = 0; g < 4; ++g) {
                    const uint4 x = *reinterpret_cast<const uint4*>(wait_place(g, 0)), y = *reinterpret_cast<const uint4*>(wait_place(g, 1));
                    const uint32_t lo[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
                    tmem_st_frag_issue(low_place(g), lo);
                }
                tmem_wait_st_all();
                tc_fence_before();
                fence_async_smem();   // K's next tile comes by TMA
                mbar_arrive(&sm.low);
            }
            ++n;
        }
        if (!ok) break;
        if (u.s_out) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float2 x = parts(s[i]);
                u.s_out[(64 * half + 2 * i) * D + row] = u.out_scale * x.x;
                u.s_out[(64 * half + 2 * i + 1) * D + row] = u.out_scale * x.y;
            }
        }
    }
    if (!ok && lane == 0) raise_status(a.ws, KDA_ERR_TIMEOUT);
}

// Few sequences, one unit a block at most: each block checks the offsets itself (cu[0] = 0, non-decreasing,
// cu[N] = T) and writes the slot it reads; blocks of one sequence write the same values. (A kernel of its own
// for it takes 5 us, against 15 for lengths 17, 33, 65 with 4 heads.)
__device__ __forceinline__ bool own_slot(const LinArgs& a) {
    const int N = a.slots, n = threadIdx.x;
    bool bad = false;
    if (n < N) {
        const int64_t from = a.cu[n], to = a.cu[n + 1];
        bad = to < from || (n == 0 && from != 0) || (n == N - 1 && to != a.T);
        if (n == (int)blockIdx.x / (a.jobs * a.H)) a.table[n] = Slot{from, (int32_t)(to - from), n, 0, 1, 0, 0};
    }
    return !__syncthreads_or(bad);
}

__global__ void __launch_bounds__(kLinThreads, 1) linattn_kernel(const __grid_constant__ LinArgs a) {
    extern __shared__ uint8_t smem_raw[];
    LinSmem& sm = *reinterpret_cast<LinSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // A call's first kernel sets the status word here, long before any wait of another CTA can give up
    // (2 s) and write to it.
    if (a.first) {
        const bool bad = a.cu && !own_slot(a);
        if (blockIdx.x == 0 && threadIdx.x == 0) *reinterpret_cast<int*>(a.ws) = bad ? KDA_ERR_OFFSETS : 0;
        if (bad) return;
    } else if (read_status(a.ws) != 0) {
        return;
    }
    const int units = units_of(a);
    const int warp = uniform((int)(threadIdx.x >> 5));
    if (warp == 0) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 32) {
        uint64_t* const one[] = {&sm.full_k[0], &sm.full_k[1], &sm.full_q, &sm.full_v[0], &sm.full_v[1], &sm.all[0], &sm.all[1],
                                 &sm.qk, &sm.qs, &sm.ds, &sm.pv, &sm.end};
        for (uint64_t* bar : one) mbar_init(bar, 1);
        uint64_t* const all_main[] = {&sm.s, &sm.piece, &sm.low, &sm.o};
        for (uint64_t* bar : all_main) mbar_init(bar, 32 * kMainWarps);
        mbar_init(&sm.p, 32 * kScoreWarps);
        mbar_init(&sm.r, 32 * kScoreWarps);
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = uniform(sm.tmem);
    if (warp < kScoreWarps) {
        lin_scores(a, sm, units, tm);
    } else if (warp < kScoreWarps + kMainWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMainRegs));
        lin_main(a, sm, units, tm);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if ((threadIdx.x & 31) == 0) {
            if (warp == kScoreWarps + kMainWarps) lin_load(a, sm, units);
            else if (warp == kScoreWarps + kMainWarps + 1) lin_mma(a, sm, units, tm);
        }
    }
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
    const int h = blockIdx.y, e = ((blockIdx.x & 15) * 256 + threadIdx.x) * 4;
    const int slots = a.slots_dev ? *a.slots_dev : a.slots;
    const float g = a.log_decay[h];
    for (int i = blockIdx.x / 16; i < slots; i += gridDim.x / 16) {
        const Slot s = slot_of(a, i);
        if (s.nseg == 1) return;   // sequences of several segments come first
        if (s.seg != 0) continue;
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
            const float over = 1.0f / j.s_scale;
            x.x *= over; x.y *= over; x.z *= over; x.w *= over;
        }
        // segments in the job's order, eight loads in flight; all but the last in time have seg_len tokens
        const int64_t step = (j.rev ? -1 : 1) * (int64_t)a.H * D * D;
        float* p = j.seg + ((size_t)(j.rev ? i + s.nseg - 1 : i) * a.H + h) * D * D + e;
        const float whole = expf(g * (float)a.seg_len), last = expf(g * (float)(s.after - (int64_t)(s.nseg - 2) * a.seg_len));
        for (int k0 = 0; k0 < s.nseg; k0 += 8, p += 8 * step) {
            float4 y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)   // the sum of the last segment in order is not there and not needed
                if (k0 + k + 1 < s.nseg) y[k] = *reinterpret_cast<const float4*>(p + k * step);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k0 + k < s.nseg) {
                    *reinterpret_cast<float4*>(p + k * step) = x;
                    if (k0 + k + 1 < s.nseg) {
                        const float w = j.rev && k0 + k == 0 ? last : whole;
                        x = make_float4(w * x.x + y[k].x, w * x.y + y[k].y, w * x.z + y[k].z, w * x.w + y[k].w);
                    }
                }
        }
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
    // sequences of several segments first, so that the states of segments take up the first places
    const int warp = tid >> 5, lane = tid & 31;
    for (int pass = seg_len < T_total ? 0 : 1; pass < 2; ++pass) {
        for (int b = 0; b < N; b += blockDim.x) {
            const int n = b + tid;
            const int64_t t0 = n < N ? cu[n] : 0, len = n < N ? cu[n + 1] - t0 : 0;
            const int cnt = n < N && (len > seg_len) == (pass == 0) ? (len > 0 ? (int)((len + seg_len - 1) / seg_len) : 1) : 0;
            int before = cnt;   // sums of the warp, then of the warps before it
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, before, o);
                if (lane >= o) before += x;
            }
            if (lane == 31) scan[warp] = before;
            __syncthreads();
            int first = carry + before - cnt, sum = 0;
            for (int w = 0; w < 32; ++w) {
                if (w == warp) first += sum;
                sum += scan[w];
            }
            for (int k = 0; k < cnt; ++k) {
                const int64_t left = len - k * seg_len;
                if (first + k < slots_max) {
                    const int32_t m = (int32_t)(left < seg_len ? left : seg_len);
                    table[first + k] = Slot{t0 + k * seg_len, m, n, k, cnt, (int32_t)(k * seg_len), (int32_t)(left - m)};
                }
            }
            __syncthreads();
            if (tid == 0) carry += sum;
            __syncthreads();
        }
    }
    if (tid == 0) {
        *slots = carry;
        *reinterpret_cast<int*>(ws) = 0;
    }
    // Whole sequences, few of them: longest first. A block's rounds come from opposite ends of the list in turn,
    // which evens them out (lengths 1300, 547, 2048, 963, 271, 3063 with 96 heads on 152 SMs: at most 46 chunks
    // on an SM instead of 59, with 43 in the mean; 215 instead of 252 us).
    if (seg_len < T_total || N > (int)blockDim.x) return;
    const Slot own = tid < N ? table[tid] : Slot{};
    scan[tid] = own.len;
    __syncthreads();
    if (tid >= N) return;
    int rank = 0;
    for (int m = 0; m < N; ++m) rank += scan[m] > own.len || (scan[m] == own.len && m < tid);
    table[rank] = own;
}

// dq, dk of a query/key head: the sum of its G value heads' shares, in head order. HBM bounds it (T = 4096, 32 heads in
// groups of 4: 21 us for 134 MB of shares). The heads of a group are on different SMs at a time, and sums in
// the order of their arrival would differ from call to call.
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
// 4 l .. 4 l + 3 of each, so that a warp moves whole 512-byte rows. 256 requests, 96 heads: 489 us, 6.6 TB/s, 99% of the
// measured copy; 4 requests, 4 heads: 9 us on the GPU, 14 with the call.
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
// sums come first (state-only units, about half of a full one's time), then the states they start
// from, then all segments at once, if that comes out shorter by the cost model. Forward, whole and as split:
// T = 4096 with 32 heads 98 and 71 us, 16384 with 8 heads 340 and 68, 1024 with 4 heads 35 and 29 (not split: 1024
// with 16 heads, 36 and 35; 4096 with 64 heads, 100 and 112); backward 16384 with 8 heads 346 and 135.
struct Plan {
    int64_t seg_len;   // tokens, a multiple of the chunk
    int nseg;          // segments of a fixed-length sequence (packed: of T_total tokens at most)
    int slots;         // fixed: slots; packed: most slots
    int kept;          // the first of them, whose states are kept in the workspace
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
        if (s > 1) t += (double)((pre * (s - 1) + kSMs - 1) / kSMs) * (kStateOnly * len + kUnitChunks) + kSplitChunks + kCarried * (double)(rows * s);
        if (s == 1 || t < least) { least = t; best = s; }
    }
    Plan p;
    p.seg_len = (chunks + best - 1) / best * LC;
    if (p.seg_len < LC) p.seg_len = LC;
    p.nseg = (int)(chunks > 0 ? (sh->T + p.seg_len - 1) / p.seg_len : 1);
    p.slots = packed ? (int)(sh->N + sh->T / p.seg_len) : (int)(sh->B * p.nseg);
    // of those, segments of sequences of several: no more than 2 (length / seg_len), rounded down, of each sequence
    p.kept = p.nseg == 1 ? 0 : packed ? (int)std::min<int64_t>(p.slots, 2 * (sh->T / p.seg_len)) : p.slots;
    return p;
}

struct LinLayout {
    Plan plan;
    size_t table, seg[2], share_q, share_k, total;
};
LinLayout layout_of(const kda_linattn_shape* sh, bool packed, bool backward) {
    const Plan p = plan_of(sh, packed, backward ? 3 : 1);
    LinLayout l;
    l.plan = p;
    size_t o = 1024;   // the status word, at byte 64 the number of slots
    l.table = o; o += packed ? align_up((size_t)p.slots * sizeof(Slot), 1024) : 0;
    const size_t states = (size_t)p.kept * sh->H * D * D * sizeof(float);
    l.seg[0] = o; o += states;
    l.seg[1] = o; o += backward ? states : 0;
    const size_t share = backward && groups_of(sh) > 1 ? align_up((size_t)(sh->B * sh->T * sh->H) * D * sizeof(float), 1024) : 0;
    l.share_q = o; o += share;
    l.share_k = o; o += share;
    l.total = o;
    return l;
}

kda_status common_checks(const kda_linattn_shape* sh, const int64_t* cu, const void* ws, size_t bytes, bool backward,
                         LinLayout* lay) {
    const kda_status st = check_shape(sh, cu != nullptr);
    if (st != KDA_OK) return st;
    *lay = layout_of(sh, cu != nullptr, backward);
    if (!ws || bytes < lay->total) return KDA_ERR_WORKSPACE;
    if (misaligned(ws) || (reinterpret_cast<uintptr_t>(cu) & 7u)) return KDA_ERR_ALIGN;
    return KDA_OK;
}

// The tensor map of a [tokens, heads, 128] bf16 (or fp32) tensor in boxes of `rows` tokens x 128 bytes.
kda_status make_map(CUtensorMap* map, const void* p, int64_t tokens, int64_t heads, int rows, bool fp32 = false) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    if (!encode) {
        set_last_error_text("the driver has no cuTensorMapEncodeTiled");
        return KDA_ERR_CUDA;
    }
    const cuuint64_t dims[3] = {D, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t size = fp32 ? 4 : 2, strides[2] = {D * size, (cuuint64_t)heads * D * size};
    const cuuint32_t box[3] = {fp32 ? 32u : 64u, 1, (cuuint32_t)rows}, step[3] = {1, 1, 1};
    const CUresult r = encode(map, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, step,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS) return KDA_OK;
    char msg[96];
    snprintf(msg, sizeof(msg), "cuTensorMapEncodeTiled: %d", (int)r);
    set_last_error_text(msg);
    return KDA_ERR_CUDA;
}

// Launches for `jobs` sums over the shape's tokens. seg[0], seg[1]: the segment states of job 0 and,
// transposed for job 1, of job 2 (the backward's two reversed jobs sum the same state).
kda_status run_jobs(const kda_linattn_shape* sh, LinArgs& a, const void* const (&tensors)[4], int jobs, const int64_t* cu, const float* log_decay, uint8_t* ws,
                    const LinLayout& lay, cudaStream_t s) {
    const Plan p = lay.plan;
    static std::atomic<uint64_t> allowed{0};   // devices on which the kernel may use its shared memory
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    const uint64_t bit = uint64_t(1) << (device & 63);
    if (e == cudaSuccess && !(allowed.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(linattn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(LinSmem) + 1024);
        if (e == cudaSuccess && device < 64) allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    if (e != cudaSuccess) {
        set_last_error_text(cudaGetErrorString(e));
        return KDA_ERR_CUDA;
    }
    const int64_t tokens = sh->B * sh->T;
    kda_status st = KDA_OK;
    for (int i = 0; i < 4 && tokens > 0 && st == KDA_OK; ++i)
        if (tensors[i]) st = make_map(&a.map[i], tensors[i], tokens, sh->H / a.group[i], LC);
    for (int i = 0; i < jobs && tokens > 0 && st == KDA_OK; ++i) {
        const LinJob& j = a.job[i];
        st = make_map(&a.out_map[i], j.share ? static_cast<void*>(j.share) : j.out, tokens, sh->H, 32, j.share != nullptr);
    }
    if (st != KDA_OK) return st;
    a.log_decay = log_decay;
    a.scale = sh->scale;
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
    Slot* const table = reinterpret_cast<Slot*>(ws + lay.table);
    if (cu && p.nseg == 1 && sh->N * sh->H * jobs <= kSMs) {
        a.cu = cu;
        a.table = table;
        a.slots = (int)sh->N;
    } else if (cu) {
        int* const slots = reinterpret_cast<int*>(ws + 64);
        linattn_table_kernel<<<1, 1024, 0, s>>>(cu, (int)sh->N, sh->T, p.seg_len, p.slots, table, slots, ws);
        a.table = table;
        a.slots_dev = slots;
        a.first = 0;
    }
    auto launch = [&](const LinArgs& x) {
        const int64_t units = (int64_t)x.slots * sh->H * x.jobs;
        linattn_kernel<<<(unsigned)(units < kSMs ? units : kSMs), kLinThreads, sizeof(LinSmem) + 1024, s>>>(x);
    };
    if (p.nseg > 1) {
        LinArgs b = a;
        b.state_only = 1;
        if (jobs > 1) { b.jobs = 2; b.job[1] = a.job[2]; }
        launch(b);
        b.first = a.first = 0;
        linattn_carry_kernel<<<dim3((unsigned)std::min(p.slots, 64) * 16, (unsigned)sh->H, (unsigned)b.jobs), 256, 0, s>>>(b);
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
            const LinLayout l = layout_of(shape, packed != 0, backward != 0);
            // the backward's workspace serves the forward too, beside the grouped gradients' shares
            const size_t share = l.total - l.share_q, f = layout_of(shape, packed != 0, false).total;
            const size_t b = (l.share_q > f ? l.share_q : f) + share;
            if (b > most) most = b;
        }
    return most;
}

extern "C" kda_status kda_linattn_fwd(const kda_linattn_shape* shape, const kda_bf16* q, const kda_bf16* k,
                                      const kda_bf16* v, const float* log_decay, const float* h0,
                                      const int64_t* cu_seqlens, kda_bf16* o, float* hT, void* workspace,
                                      size_t workspace_bytes, void* stream) {
    LinLayout lay;
    const kda_status st = common_checks(shape, cu_seqlens, workspace, workspace_bytes, false, &lay);
    if (st != KDA_OK) return st;
    if ((shape->B * shape->T > 0 && (!q || !k || !v || !o)) || !log_decay) return KDA_ERR_NULL;
    const void* ptrs[] = {q, k, v, log_decay, h0, o, hT};
    for (const void* p : ptrs)
        if (misaligned(p)) return KDA_ERR_ALIGN;
    const int G = groups_of(shape);
    LinArgs a{{}, {}, {G, G, 1, 1}};
    a.job[0] = LinJob{0, 1, 2, o, nullptr, h0, hT, nullptr, 0, 0, 0, hT != nullptr, 1.0f};
    const kda_status rs = run_jobs(shape, a, {q, k, v, nullptr}, 1, cu_seqlens, log_decay, static_cast<uint8_t*>(workspace),
                                   lay, static_cast<cudaStream_t>(stream));
    return rs != KDA_OK ? rs : launched("kda_linattn_fwd launch");
}

extern "C" kda_status kda_linattn_bwd(const kda_linattn_shape* shape, const kda_bf16* q, const kda_bf16* k,
                                      const kda_bf16* v, const float* log_decay, const float* h0,
                                      const int64_t* cu_seqlens, const kda_bf16* do_, const float* dhT, kda_bf16* dq,
                                      kda_bf16* dk, kda_bf16* dv, float* dh0, void* workspace, size_t workspace_bytes,
                                      void* stream) {
    LinLayout lay;
    const kda_status st = common_checks(shape, cu_seqlens, workspace, workspace_bytes, true, &lay);
    if (st != KDA_OK) return st;
    const int64_t tokens = shape->B * shape->T;
    if ((tokens > 0 && (!q || !k || !v || !do_ || !dq || !dk || !dv)) || !log_decay) return KDA_ERR_NULL;
    const void* ptrs[] = {q, k, v, log_decay, h0, do_, dhT, dq, dk, dv, dh0};
    for (const void* p : ptrs)
        if (misaligned(p)) return KDA_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const int G = groups_of(shape);
    float* const share_q = G > 1 ? reinterpret_cast<float*>(ws + lay.share_q) : nullptr;
    float* const share_k = G > 1 ? reinterpret_cast<float*>(ws + lay.share_k) : nullptr;
    const float sc = shape->scale;
    LinArgs a{{}, {}, {G, G, 1, 1}};
    a.job[0] = LinJob{3, 2, 1, dq, share_q, h0, nullptr, nullptr, 1, 0, 0, 0, 1.0f};
    a.job[1] = LinJob{2, 3, 0, dk, share_k, dhT, nullptr, nullptr, 1, 1, 1, 0, sc};
    a.job[2] = LinJob{1, 0, 3, dv, nullptr, dhT, dh0, nullptr, 0, 0, 1, dh0 != nullptr, sc};
    const kda_status rs = run_jobs(shape, a, {q, k, v, do_}, 3, cu_seqlens, log_decay, ws, lay, s);
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
