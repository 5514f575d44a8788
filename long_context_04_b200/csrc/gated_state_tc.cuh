// The state scan of gated lightning attention on the tensor cores (bf16 inputs).
//
//   forward   X = state at a block's start,        X <- e^{G_C} X + sum_j k_j (e^{G_C - G_j} v_j)^T
//   reverse   X = state gradient at its end,       X <- e^{G_C} X + sum_i q_i (e^{G_i} do_i)^T
//
// over blocks of C = 128 tokens; the value of X before each update goes to a snapshot per block,
// from which the block kernels then run independently of each other.  A snapshot is an operand
// of bf16 products, so it is left as two bf16 parts, the second the rounding of what the first
// leaves (16 bits).  One part would do for vectors of D entries, but not for the gate's gradient,
// one number per token and head whose terms <dS, S>, q . S do and k . dS v may cancel: with it
// a fifth to two fifths of the heads of up to 1000 tokens with a long memory were off by more
// than 1.5 times the rounding of the result, some by eight times; with two parts it is the
// rounding alone.  They cost their traffic: 8192 tokens, 64 heads, D = 128, the two scans together 249 us
// instead of 206.  X itself stays fp32 from block to block.
//
// One CTA per (segment, head, 64-column slice of the state).  Per block the tile of the left
// factor (128 x D) and the slice of the right one (128 x 64) arrive by TMA; eight warps scale
// the slice's rows by their decays and split every product into three bf16 numbers whose sum
// is the fp32 product to 2^-26 (one bf16 alone would round the state by 2^-9 in every step);
// one warp issues the product of the tile with the first two parts side by side (one read of
// the left factor from shared memory for both) and adds that with the third to the second's
// columns, a quarter of the tokens at a time as they are scaled; the epilogue adds the two
// accumulators to the fp32 state in its registers and stores the snapshots by TMA.
//
// The tensor work (3 x 2 D^2 flops per token) is below its HBM time: 4 D bytes read (the left
// tile is read by D / 64 CTAs, mostly from L2) and 4 D^2 / 128 bytes of snapshot written per
// token and head; the reverse scan reads as many bytes of forward snapshots again.  At 8192
// tokens, 64 heads, D = 128 the forward scan takes 105 us (537 MB, 5.1 TB/s; 1.64 us a block),
// bound by the chain of one block after the other, and the reverse one 144 us (805 MB, 5.6 TB/s,
// 85 % of the copy rate), the tensor cores of its 128 SMs busy for 28 and 21 % of it.
//
// Warpgroups (640 threads; registers are moved to those that hold the state):
//   0  warp 0 loads of the tiles; warp 1 MMA issue; warp 2 gate sums; warp 3 loads of the forward
//      snapshots (reverse scan)
//   1, 2  epilogue, 32 columns each: the state, its snapshots, in the reverse scan the parts of
//      e^{G_C} <X, state>.  (Before snapshots had two parts, one warpgroup for all 64 columns cost
//      the two scans together 7 us.)
//   3, 4  scaling.  (At that time a backward call took 464 us, with one warpgroup 510.)
// Three slots for the tiles: with two the next tile came too late (446 and 464 us).  The reverse scan at D = 128 has room for two slices of 64 columns only.
#pragma once

#include "gated.cuh"

namespace la {

struct GatedStateParams {
    CUtensorMap tmap_a;         // k (forward) or q (reverse): [T][H*D], box 64 x 128
    CUtensorMap tmap_b;         // v or do
    const __nv_bfloat16 *g;     // [T][H] or nullptr
    const float *initial;       // [S][H][D][D] or nullptr
    const float *seg_in;        // [segs][H][D][D]: start states of a segmented call, or nullptr
    float *seg_out;             // [segs][H][D][D]: a segment's own end state, or nullptr
    float *seg_total;           // [segs][H]: its summed log-decay
    float *fin;                 // [S][H][D][D] or nullptr: final states
    CUtensorMap tmap_snap;      // snapshots, [blocks * H][2 parts][D][D], box 64 x D
    CUtensorMap tmap_other;     // reverse: the forward snapshots, the same
    int have_snap;
    float *through;             // reverse: [blocks][H][8 D / 64] parts of e^{G_C} <X, state>, or nullptr
    int H;
    unsigned long long timeout_ns;
    GatedTable tab;
};

template <int D, bool REV>
struct GatedStateCfg {
    static constexpr int C = 128;
    static constexpr int NVS = D / 64;              // column slices (CTAs) per (segment, head)
    static constexpr int DB = D / 64;               // 64-column boxes of the left tile
    static constexpr int BOX = C * 128;             // 128 rows x 128 B
    static constexpr int SBOX = D * 128;            // a slice of a state's snapshot
    static constexpr int TILE = DB * BOX;           // the left tile
    static constexpr int NST = 3, NSB = REV && D == 128 ? 2 : 3;  // slots for left tiles, for slices
    static constexpr int OFF_B = NST * TILE;        // slices (later their first part)
    static constexpr int OFF_PARTS = OFF_B + NSB * BOX;                   // the slice's second and third parts
    static constexpr int OFF_SNAP = OFF_PARTS + 2 * BOX;                  // a snapshot's parts on their way out
    static constexpr int OFF_OTHER = OFF_SNAP + 2 * SBOX;                 // reverse: a forward snapshot's parts
    static constexpr int OFF_G = OFF_OTHER + (REV ? 2 * SBOX : 0);           // gate sums, two blocks
    static constexpr int OFF_MISC = OFF_G + 2 * C * 4;
    static constexpr int SMEM_BYTES = 1024 + OFF_MISC + 512;
    static_assert(SMEM_BYTES > 114 * 1024 && SMEM_BYTES <= 227 * 1024, "one CTA per SM");
    static constexpr int TMEM_COLS = 256;           // two accumulators of 128 columns
    static constexpr int ACC = 128;
    static constexpr int GROUP = 256, THREADS = 128 + 2 * GROUP;  // threads of the epilogue, of scaling
    // registers a thread: launched with 96; the shares of the five warpgroups add up to 5 * 96
    static constexpr int R_LAUNCH = 96, R_MISC = 56, R_STATE = 128, R_SCALE = 80;
    static_assert(R_MISC + 2 * R_STATE + 2 * R_SCALE <= 5 * R_LAUNCH, "register shares");
    static constexpr uint32_t ID2 = idesc_bf16_f32(D, 128, 1, 1), ID1 = idesc_bf16_f32(D, 64, 1, 1);
};

struct GatedStateMisc {
    uint64_t full[3], empty[3];            // tiles landed, released
    uint64_t ready[4], parts_free[4];      // a quarter of the slice scaled, multiplied
    uint64_t acc_full[2], acc_free[2];
    uint64_t other_full, other_free;       // reverse: the forward snapshot of a block
    uint64_t gates_ready[2], gates_free[2];
    uint64_t done;
    float sum[2];          // log-decay of a block, times log2(e)
    uint32_t tmem_base;
    int abort_flag;
};

template <int N>
__device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// A wait of a whole warp for a phase: true once every lane has seen it complete, false after
// `limit_ns` or once another warp gave up.  Written for few instructions: these kernels run
// six roles at once, whose code has to fit the instruction cache together.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const volatile int *abort_flag,
                                          uint64_t limit_ns) {
    const uint32_t addr = smem_u32(bar);
    uint64_t t0 = 0;
#pragma unroll 1
    while (!__all_sync(0xffffffffu, mbar_try_wait(addr, parity))) {
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (__any_sync(0xffffffffu, *abort_flag != 0 || now - t0 > limit_ns)) return false;
    }
    return true;
}

// The log-decays of tokens 4 * lane .. 4 * lane + 3 of a block, as they lie in memory (0
// behind the sequence), and as the kernels use them.  Fetched a block ahead: the widening
// is kept behind what the caller waits for in between, or the loads' latency would be
// waited for at once.
__device__ __forceinline__ void fetch_gates4(uint32_t (&raw)[4], const __nv_bfloat16 *__restrict__ g, int row0,
                                             int nv, int H, int h) {
    const int lane = threadIdx.x & 31;
    const unsigned short *src = reinterpret_cast<const unsigned short *>(g) + (size_t)(row0 + 4 * lane) * H + h;
#pragma unroll
    for (int e = 0; e < 4; ++e) raw[e] = g != nullptr && 4 * lane + e < nv ? src[(size_t)e * H] : 0u;
}
__device__ __forceinline__ void widen_gates4(float (&x)[4], uint32_t (&raw)[4]) {
    asm volatile("" : "+r"(raw[0]), "+r"(raw[1]), "+r"(raw[2]), "+r"(raw[3]));
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = clamp_gate(__uint_as_float(raw[e] << 16));
}

// Sums from the block's start up to and including each of the lane's four tokens; returns
// the sum over the block.
__device__ __forceinline__ float prefix_gates4(const float (&x)[4], float (&sum)[4]) {
    const int lane = threadIdx.x & 31;
    sum[0] = x[0];
    sum[1] = sum[0] + x[1];
    sum[2] = sum[1] + x[2];
    sum[3] = sum[2] + x[3];
    float run = sum[3];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const float y = __shfl_up_sync(0xffffffffu, run, off);
        if (lane >= off) run += y;
    }
    float before = __shfl_up_sync(0xffffffffu, run, 1);
    if (lane == 0) before = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] += before;
    return __shfl_sync(0xffffffffu, run, 31);
}

// Sums over the tokens behind each of the lane's four tokens, up to the block's end: summed
// from the end, so that a decay near 1 comes from a short, exact sum.
__device__ __forceinline__ float suffix_gates4(const float (&x)[4], float (&sum)[4]) {
    const int lane = threadIdx.x & 31;
    const float own = (x[3] + x[2]) + (x[1] + x[0]);
    float run = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const float y = __shfl_down_sync(0xffffffffu, run, off);
        if (lane + off < 32) run += y;
    }
    float after = __shfl_down_sync(0xffffffffu, run, 1);
    if (lane == 31) after = 0.f;
    sum[3] = after;
    sum[2] = after + x[3];
    sum[1] = sum[2] + x[2];
    sum[0] = sum[1] + x[1];
    return __shfl_sync(0xffffffffu, run, 0);
}

// Products, sums and differences of fp32 pairs.
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint32_t pack_f32x2(uint64_t x) {  // two fp32 values as a bf16 pair
    uint32_t lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(x));
    return pack_bf16x2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint64_t sub_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t pair_f32(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
// The two values of a bf16 pair as fp32.
__device__ __forceinline__ uint64_t widen_bf16x2(uint32_t x) { return pair_f32(x << 16, x & 0xffff0000u); }

// One 16-byte chunk of eight bf16 values scaled by w, as PARTS bf16 numbers each, every one
// the rounding of what the earlier ones leave.  `keep` false gives zeros whatever the chunk holds.
template <int PARTS>
__device__ __forceinline__ void split_chunk(const uint4 &raw, float w, bool keep, uint4 (&part)[PARTS]) {
    const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
    const uint64_t ww = pair_f32(__float_as_uint(w), __float_as_uint(w));
    uint32_t out[PARTS][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint64_t x = mul_f32x2(ww, widen_bf16x2(keep ? in[e] : 0u));
#pragma unroll
        for (int y = 0; y < PARTS; ++y) {
            out[y][e] = pack_f32x2(x);
            if (y + 1 < PARTS) x = sub_f32x2(x, widen_bf16x2(out[y][e]));
        }
    }
#pragma unroll
    for (int y = 0; y < PARTS; ++y) part[y] = make_uint4(out[y][0], out[y][1], out[y][2], out[y][3]);
}

__device__ __forceinline__ uint4 pack_chunk(const float *x) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// Eight fp32 values as two bf16 parts, the second the rounding of what the first leaves: 16 bits.
__device__ __forceinline__ void two_parts(const float *x, uint4 (&part)[2]) {
    uint32_t out[2][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint64_t v = pair_f32(__float_as_uint(x[2 * e]), __float_as_uint(x[2 * e + 1]));
        out[0][e] = pack_f32x2(v);
        out[1][e] = pack_f32x2(sub_f32x2(v, widen_bf16x2(out[0][e])));
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) part[y] = make_uint4(out[y][0], out[y][1], out[y][2], out[y][3]);
}

// What the kernels keep of a block's log-decays, in shared memory, times log2(e): for token i
// the sum over the tokens behind it, s_i = g_{i+1} + .. + g_{C-1}, and the sum over the block.
// Then e^{G_C - G_j} = 2^{s_j}, e^{G_i - G_j} = 2^{s_j - s_i}, e^{G_i} = 2^{sum - s_i}.  The
// reverse scan (PREFIX) keeps the sums up to and including token i instead.  Either is summed
// from the end at which the state's weights are near 1, so that those come from short sums
// and the fp32 state loses nothing to a difference of two long ones.
// Written by one warp, lane l the tokens 4 l .. 4 l + 3: a gate is one 2-byte word per row of
// H, and read by every warp on its own it cost 32 passes of the memory pipe per load.
template <bool PREFIX = false>
__device__ __forceinline__ void store_gate_sums(float *s, float *sum, const float (&x)[4]) {
    constexpr float kLog2e = 1.4426950408889634f;
    const int lane = threadIdx.x & 31;
    float y[4];
    const float all = PREFIX ? prefix_gates4(x, y) : suffix_gates4(x, y);
    *reinterpret_cast<float4 *>(&s[4 * lane]) = make_float4(y[0] * kLog2e, y[1] * kLog2e, y[2] * kLog2e, y[3] * kLog2e);
    if (lane == 0) *sum = all * kLog2e;
}

// 2^x of both values of a pair.
__device__ __forceinline__ uint64_t ex2_f32x2(uint64_t x) {
    uint64_t r;
    asm("{\n\t.reg .f32 a, b;\n\t"
        "mov.b64 {a, b}, %1;\n\t"
        "ex2.approx.ftz.f32 a, a;\n\t"
        "ex2.approx.ftz.f32 b, b;\n\t"
        "mov.b64 %0, {a, b};\n\t}"
        : "=l"(r)
        : "l"(x));
    return r;
}

// 16 consecutive TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// MMA issue by a whole converged warp, of which `leader` (elected once) is true in one lane:
// the descriptors stay warp-uniform values, which one lane's branch would have to move over
// one by one in front of every instruction.
__device__ __forceinline__ uint32_t elect_leader() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r;
}
__device__ __forceinline__ void warp_mma_ss(uint32_t leader, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void warp_mma_ts(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void warp_commit(uint32_t leader, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(leader)
        : "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 r;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "r"(addr));
    return r;
}
// What this thread has read from shared memory so far has been read: behind it an arrival may
// give the place to other threads' ordinary stores.  (An arrival releases ordinary accesses of
// its own thread; where lane 0 arrives for its warp, the others' reads come before it through
// this and __syncwarp.)  A place that TMA or a product's operands take next needs
// fence_proxy_async_smem instead: the barrier does not order ordinary reads with the async
// proxy's writes, and rows were seen to be loaded after their place had been refilled.
__device__ __forceinline__ void reads_done() { __threadfence_block(); }
__device__ __forceinline__ void st_shared_u4(uint32_t addr, const uint4 &v) {
    st_shared_v4(addr, v.x, v.y, v.z, v.w);
}

template <int D, bool REV>
__global__ void __launch_bounds__(GatedStateCfg<D, REV>::THREADS, 1)
    gated_state_tc_kernel(const __grid_constant__ GatedStateParams p) {
    using C = GatedStateCfg<D, REV>;
    static_assert(sizeof(GatedStateMisc) <= 512, "misc area");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    GatedStateMisc *m = reinterpret_cast<GatedStateMisc *>(smem + C::OFF_MISC);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int vs = blockIdx.x % C::NVS;
    const int h = (blockIdx.x / C::NVS) % p.H, sg = blockIdx.x / (C::NVS * p.H);
    int rank, s, start, len, sid;
    p.tab.seg(sg, rank, s);
    p.tab.seqs.get(rank, start, len, sid);
    const int all = (len + C::C - 1) / C::C;
    const int b0 = s * p.tab.seg_blocks, nb = max(0, min(all, b0 + p.tab.seg_blocks) - b0);
    const int first = p.tab.first_block(rank);
    const bool through = REV && p.through != nullptr;
    const uint64_t tlimit = p.timeout_ns;
    volatile int *abort_flag = &m->abort_flag;
    // the t-th block that the scan visits, its tokens, its number (times H, plus h) in the call
    auto block_of = [&](int t) { return REV ? b0 + nb - 1 - t : b0 + t; };
    auto rows_of = [&](int t) { return min(C::C, len - block_of(t) * C::C); };
    auto number_of = [&](int t) { return (first + block_of(t)) * p.H + h; };

    if (threadIdx.x == 0) {
        for (int i = 0; i < 3; ++i) {
            mbar_init(&m->full[i], 1);
            mbar_init(&m->empty[i], 1);
        }
        for (int u = 0; u < 4; ++u) {
            mbar_init(&m->ready[u], 64);
            mbar_init(&m->parts_free[u], 1);
        }
        mbar_init(&m->other_full, 1);
        mbar_init(&m->other_free, C::GROUP);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m->acc_full[i], 1);
            mbar_init(&m->acc_free[i], C::GROUP);
            mbar_init(&m->gates_ready[i], 32);
            mbar_init(&m->gates_free[i], 16);  // the warps of the epilogue and of scaling
        }
        mbar_init(&m->done, 1);
        m->abort_flag = 0;
        fence_mbarrier_init_cluster();
        tma_prefetch_desc(&p.tmap_a);
        tma_prefetch_desc(&p.tmap_b);
    }
    if (warp == 1) {
        tmem_alloc(&m->tmem_base, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = m->tmem_base;
    next_may_start();
    previous_done();
    auto fail = [&]() {
        *abort_flag = 1;
        record_fault(DEV_TIMEOUT);
    };
    auto wwait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return warp_wait(bar, parity, abort_flag, tlimit);
    };
    // Parity of use t of a ring of one, two or three slots; a slot is used again only after the
    // release of its last use, so that each wait below sees the phase it means.
    auto one = [](int t) { return (uint32_t)(t & 1); };
    auto two = [](int t) { return (uint32_t)((t >> 1) & 1); };
    auto three = [](int t) { return (uint32_t)((t / 3) & 1); };
    auto tile_at = [&](int t) { return sbase + (uint32_t)((t % 3) * C::TILE); };
    auto slice_at = [&](int t) { return sbase + C::OFF_B + (uint32_t)((t % C::NSB) * C::BOX); };

    if (warp < 4) {
        reg_dec<C::R_MISC>();
        bool ok = true;
        if (warp == 0) {
            // ------------------------------------------------------------ loads of the tiles
            int issued = 0;
            for (int t = 0; t < nb; ++t) {
                if (!(ok = wwait(&m->empty[t % 3], three(t) ^ 1u))) break;
                const int row = start + block_of(t) * C::C, col = h * D;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&m->full[t % 3], (uint32_t)(C::TILE + C::BOX));
#pragma unroll
                    for (int d = 0; d < C::DB; ++d)
                        tma_load_2d(tile_at(t) + d * C::BOX, &p.tmap_a, col + 64 * d, row, &m->full[t % 3]);
                    if (C::NSB < 3) tma_prefetch_l2_2d(&p.tmap_b, col + 64 * vs, row);
                }
                ++issued;
                // with two slots for slices, the last but one's products have to be done too (their
                // next phase needs the tile of t + 1)
                if (C::NSB < 3 && t >= 2 && !(ok = wwait(&m->empty[(t - 2) % 3], three(t - 2)))) break;
                if (lane == 0) tma_load_2d(slice_at(t), &p.tmap_b, col + 64 * vs, row, &m->full[t % 3]);
            }
            if (!ok) fail();
            // loads that are still in flight land before the CTA ends
            for (int t = max(0, issued - 3); t < issued; ++t)
                mbar_wait(&m->full[t % 3], three(t), nullptr, tlimit);
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issue
            const uint32_t leader = elect_leader();
            for (int t = 0; ok && t < nb; ++t) {
                ok = wwait(&m->full[t % 3], three(t)) && (t < 2 || wwait(&m->acc_free[t & 1], two(t - 2)));
                // [dims][2 x 64 columns] = A^T [part 0 | part 1 + part 2]
                const uint32_t b = slice_at(t), parts = sbase + C::OFF_PARTS;
                const uint64_t ad = desc_mnmajor_sw128(tile_at(t), C::BOX);
                const uint64_t bd = desc_mnmajor_sw128(b, parts - b), ld = desc_mnmajor_sw128(parts + C::BOX, C::BOX);
                const uint32_t acc = tmem + C::ACC * (t & 1);
#pragma unroll 1
                for (int u = 0; u < 4; ++u) {
                    // ready of t + 1 needs parts_free of t
                    if (!ok || !(ok = wwait(&m->ready[u], one(t)))) break;
                    tc_fence_after();
#pragma unroll
                    for (int ks = 2 * u; ks < 2 * u + 2; ++ks)
                        warp_mma_ss(leader, acc, desc_add(ad, ks * 2048), desc_add(bd, ks * 2048), C::ID2,
                                    ks > 0 ? 1u : 0u);
#pragma unroll
                    for (int ks = 2 * u; ks < 2 * u + 2; ++ks)
                        warp_mma_ss(leader, acc + 64, desc_add(ad, ks * 2048), desc_add(ld, ks * 2048), C::ID1, 1u);
                    warp_commit(leader, &m->parts_free[u]);
                }
                if (ok) {
                    warp_commit(leader, &m->empty[t % 3]);
                    warp_commit(leader, &m->acc_full[t & 1]);
                }
            }
            if (!ok) fail();
            warp_commit(leader, &m->done);  // every issued MMA has finished before TMEM is freed
            mbar_wait(&m->done, 0u, nullptr, tlimit);
        } else if (warp == 2) {
            // ------------------------------------------------------------ gate sums
            uint32_t raw[4];
            float gate[4];
            auto fetch = [&](int t) {
                fetch_gates4(raw, p.g, start + block_of(t) * C::C, rows_of(t), p.H, h);
            };
            if (nb > 0) fetch(0);
            for (int t = 0; t < nb; ++t) {
                if (!(ok = wwait(&m->gates_free[t & 1], two(t) ^ 1u))) break;
                widen_gates4(gate, raw);
                store_gate_sums<REV>(reinterpret_cast<float *>(smem + C::OFF_G) + C::C * (t & 1), &m->sum[t & 1], gate);
                mbar_arrive(&m->gates_ready[t & 1]);
                if (t + 1 < nb) fetch(t + 1);
            }
            if (!ok) fail();
        } else if (through) {
            // ------------------------------------------------------------ forward snapshots
            for (int t = 0; t < nb; ++t) {
                if (!(ok = wwait(&m->other_free, one(t) ^ 1u))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&m->other_full, (uint32_t)(2 * C::SBOX));
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        tma_load_2d(sbase + C::OFF_OTHER + y * C::SBOX, &p.tmap_other, 64 * vs,
                                    (2 * number_of(t) + y) * D, &m->other_full);
                        if (t + 1 < nb) tma_prefetch_l2_2d(&p.tmap_other, 64 * vs, (2 * number_of(t + 1) + y) * D);
                    }
                }
                __syncwarp();
                // the epilogue frees the place only once this load has landed; the last one:
                if (t == nb - 1) mbar_wait(&m->other_full, one(t), nullptr, tlimit);
            }
            if (!ok) fail();
        }
        __syncwarp();
    } else if (warp < 12) {
        // ---------------------------------------------------------------- epilogue: the state
        reg_inc<C::R_STATE>();
        const int q = warp & 3;
        // row i of the accumulators: lane i for M = 128; lanes 0..15 of each 32-lane
        // quadrant for M = 64
        const int i = D == 128 ? 32 * q + lane : 16 * q + lane;
        const bool i_ok = D == 128 || lane < 16;
        const uint32_t lane_base = (uint32_t)(32 * q) << 16;
        const int cg = (warp - 4) >> 2, col = 64 * vs + 32 * cg;  // this thread's columns of the state
        float X[32];  // X[i][col .. col + 31]
#pragma unroll
        for (int x = 0; x < 32; ++x) X[x] = 0.f;
        const float *from = nullptr;
        if (p.seg_in != nullptr)
            from = p.seg_in + ((size_t)sg * p.H + h) * D * D;
        else if (p.initial != nullptr)
            from = p.initial + ((size_t)sid * p.H + h) * D * D;
        if (from != nullptr && i_ok) {
            const float4 *src = reinterpret_cast<const float4 *>(from + (size_t)i * D + col);
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const float4 f = src[x];
                X[4 * x] = f.x, X[4 * x + 1] = f.y, X[4 * x + 2] = f.z, X[4 * x + 3] = f.w;
            }
        }
        float total = 0.f;
        bool ok = true;
        // After a failed wait a warp goes on through the blocks without doing anything but meeting
        // the others at the named barriers, so that none waits there for ever.
        for (int t = 0; t < nb; ++t) {
            // gates_ready of t + 2 needs this warp's gates_free of t
            if (ok) ok = wwait(&m->gates_ready[t & 1], two(t));
            const float G = m->sum[t & 1], decay = exp2f(G);
            if (ok) {
                reads_done();
                __syncwarp();
                if (lane == 0) mbar_arrive(&m->gates_free[t & 1]);
                total += G;
            }
            if (ok && through) {
                // part of e^{G_C} <X, state at the block's start>: this warp's rows and columns.
                // other_full of t + 1 needs other_free of t.
                ok = wwait(&m->other_full, one(t));
                const uint32_t at = sbase + C::OFF_OTHER + (i_ok ? i : 0) * 128;
                float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t c = at + (((4 * cg + x) ^ (i & 7)) << 4);
                    const uint4 hi = ld_shared_v4(c), lo = ld_shared_v4(c + C::SBOX);
                    const uint32_t in[4] = {hi.x, hi.y, hi.z, hi.w}, rest[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x0 = X[8 * x + 2 * e], x1 = X[8 * x + 2 * e + 1];
                        part[e] = fmaf(__uint_as_float(in[e] << 16), x0, part[e]);
                        part[e] = fmaf(__uint_as_float(in[e] & 0xffff0000u), x1, part[e]);
                        part[e] = fmaf(__uint_as_float(rest[e] << 16), x0, part[e]);
                        part[e] = fmaf(__uint_as_float(rest[e] & 0xffff0000u), x1, part[e]);
                    }
                }
                float f = i_ok ? (part[0] + part[1]) + (part[2] + part[3]) : 0.f;
                if (ok) {
                    fence_proxy_async_smem();  // the rows have been read, and TMA may write
                    mbar_arrive(&m->other_free);
                }
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) f += __shfl_xor_sync(0xffffffffu, f, off);
                if (ok && lane == 0)
                    p.through[(size_t)number_of(t) * (8 * C::NVS) + 8 * vs + 4 * cg + q] = decay * f;
            }
            if (p.have_snap) {
                // the parts' rows into their place, which the stores of the block before have read; then
                // one thread stores the slice
                if (warp == 4 && lane == 0) bulk_wait_read_all();
                __syncwarp();
                named_barrier(1, C::GROUP);
                const uint32_t at = sbase + C::OFF_SNAP;
                if (i_ok) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        uint4 part[2];
                        two_parts(&X[8 * x], part);
                        const uint32_t c = at + i * 128 + (((4 * cg + x) ^ (i & 7)) << 4);
                        st_shared_u4(c, part[0]);
                        st_shared_u4(c + C::SBOX, part[1]);
                    }
                }
                fence_proxy_async_smem();
                named_barrier(1, C::GROUP);
                if (ok && warp == 4 && lane == 0) {
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        tma_store_2d(&p.tmap_snap, at + y * C::SBOX, 64 * vs, (2 * number_of(t) + y) * D);
                    bulk_commit_group();
                }
                __syncwarp();
            }
            if (ok) ok = wwait(&m->acc_full[t & 1], two(t));
            if (ok) {
                tc_fence_after();
                const uint32_t tA = tmem + C::ACC * (t & 1) + 32 * cg + lane_base;
                uint32_t a[32], c[32];
                tmem_ld32(tA, a);
                tmem_ld32(tA + 64, c);
                tmem_ld_wait();
                tc_fence_before();
                mbar_arrive(&m->acc_free[t & 1]);
#pragma unroll
                for (int z = 0; z < 32; ++z)
                    X[z] = fmaf(decay, X[z], __uint_as_float(a[z]) + __uint_as_float(c[z]));
            }
        }
        if (warp == 4 && lane == 0) bulk_wait_all();
        float *to = nullptr;
        if (p.seg_out != nullptr)
            to = p.seg_out + ((size_t)sg * p.H + h) * D * D;
        else if (p.fin != nullptr && s == (REV ? 0 : p.tab.num_segs(rank) - 1))
            to = p.fin + ((size_t)sid * p.H + h) * D * D;
        if (ok && to != nullptr && i_ok) {
            float4 *d4 = reinterpret_cast<float4 *>(to + (size_t)i * D + col);
#pragma unroll
            for (int x = 0; x < 8; ++x) d4[x] = make_float4(X[4 * x], X[4 * x + 1], X[4 * x + 2], X[4 * x + 3]);
        }
        if (ok && p.seg_out != nullptr && vs == 0 && warp == 4 && lane == 0)
            p.seg_total[(size_t)sg * p.H + h] = total * 0.6931471805599453f;
        if (!ok) fail();
    } else {
        // ---------------------------------------------------------------- scaling: 16 rows a warp
        reg_dec<C::R_SCALE>();
        const int w8 = warp - 12, u = w8 >> 1;
        bool ok = true;
        for (int t = 0; t < nb; ++t) {
            const int nv = rows_of(t);
            const float *sg2 = reinterpret_cast<const float *>(smem + C::OFF_G) + C::C * (t & 1);
            // parts_free of t needs ready of t
            if (!wwait(&m->gates_ready[t & 1], two(t)) || !wwait(&m->full[t % 3], three(t)) ||
                (t >= 1 && !wwait(&m->parts_free[u], one(t - 1)))) {
                ok = false;
                break;
            }
            const uint32_t b = slice_at(t), parts = sbase + C::OFF_PARTS;
            // chunk c of row r lies in one of the row's eight 16-byte places, whichever the
            // swizzle says; all eight are scaled alike
#pragma unroll 2
            for (int x = 0; x < 4; ++x) {
                const int c = w8 * 128 + x * 32 + lane, r = c >> 3;
                uint4 part[3];
                split_chunk(ld_shared_v4(b + c * 16), exp2f(sg2[r]), r < nv, part);
                st_shared_u4(b + c * 16, part[0]);
                st_shared_u4(parts + c * 16, part[1]);
                st_shared_u4(parts + C::BOX + c * 16, part[2]);
            }
            // rows of another sequence: 0 times what they hold could be a NaN
            for (int c = max(nv, 16 * w8) * 8 + lane; c < (16 * w8 + 16) * 8; c += 32)
                for (int d = 0; d < C::DB; ++d) st_shared_v4(tile_at(t) + d * C::BOX + c * 16, 0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            mbar_arrive(&m->ready[u]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&m->gates_free[t & 1]);
        }
        if (!ok) fail();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

}  // namespace la
