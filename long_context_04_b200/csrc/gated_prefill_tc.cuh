// Gated lightning-attention prefill on the tensor cores (bf16): TMA + tcgen05 + TMEM.
//
// Per block of 128 tokens of one sequence and head (G, S as in gated.cuh):
//     o  = [(q k^T) (.) e^{G_i - G_j}, j <= i] v  +  e^{G_i} (q S)
//     S <- e^{G_C} S + k^T (e^{G_C - G_j} v_j)
// One CTA runs the blocks of one (segment, head, 64-column slice of v and o) in order, with
// the state on chip: every q, k, v is read once and every o written once.
//
// Products per block: scores q k^T (128 x 128), q S, P v (128 x 64 each, into accumulators of
// their own: their rows are scaled apart), and k^T v' with v' the decayed values split into
// three bf16 parts (see gated_state_tc.cuh): one product of two parts side by side, [part 0 |
// part 1], and one that adds part 2 to part 1's columns.
// P goes back to TMEM over the scores it came from and is read there as the left factor.  P and
// the state's snapshot are one bf16 number each, as operands of products whose results are
// vectors of D entries: o is off by 2.3e-3 instead of 1.7e-3, and its norm does not cancel.
//
// Warpgroups (768 threads; registers are moved to the group that holds the state):
//   0  warp 0 TMA loads; three issuers: warp 1 the scores, warp 2 q S and P v, warp 3 k^T v'
//   1  group KV: the fp32 state in registers, its bf16 snapshot for q S, the final state
//   2  group P: scores -> decay, mask -> P
//   3  group O: e^{G_i} (q S) + P v -> bf16 -> global
//   4, 5  group V: v -> v', zeros behind the sequence's end
// q, k and v have rings of two slots each, released by their last readers, so that the next
// block's scores and k^T v' run while this block's output is still being formed.
//
// The two slices of a head are two CTAs because TMEM has no room for two scores, q S, P v and
// the state's increments (two parts) over all 128 columns; they read q and k twice, the second
// time from L2 (404 MB of DRAM reads for 403 MB of q, k, v).
//
// Limits per block and CTA at D = 128: HBM 64 KB of a pair's 128 KB (2360 cycles of the
// measured copy rate over 128 CTAs), tensor 1900 cycles, shared memory about 2900 cycles
// (tiles in, operands out, v' written and read).  Measured: 8192 tokens, 64 heads 165 us,
// 16384 299 us (2.3 us or 4400 cycles a block; 3.6 TB/s), tensor cores busy for 36 % of it,
// issue slots for 48 %.  The chain scores -> P -> P v -> output of a block bounds it, not one
// unit.  What did not help: v' in two parts instead of three (-5 %, and the state would carry
// rounding of 2^-17), q S and P v as one product behind P (+3 %), e^{G_i} and e^{-G_j} as
// factors (0 to +1.5 %), a third slot for v (+2 %), polling by one lane (+50 %).
#pragma once

#include "gated_state_tc.cuh"

namespace la {

struct GatedPrefillParams {
    CUtensorMap tmap_q, tmap_k, tmap_v;   // [T][H*D], box 64 x 128
    CUtensorMap tmap_o;                   // o, box 64 x 32
    const __nv_bfloat16 *g;
    __nv_bfloat16 *o;
    const float *initial;                 // as in GatedStateParams
    const float *seg_in;
    float *fin;
    int H;
    unsigned long long timeout_ns;
    GatedTable tab;
};

template <int D>
struct GatedPrefillCfg {
    static constexpr int C = 128;
    static constexpr int PARTS = 3;                    // bf16 numbers for a decayed value
    static constexpr int NVS = D / 64;
    static constexpr int DB = D / 64;
    static constexpr int BOX = C * 128;
    static constexpr int TILE = DB * BOX;              // q or k
    static constexpr int OFF_Q = 0, OFF_K = 2 * TILE, OFF_V = 4 * TILE;
    static constexpr int OFF_VP = OFF_V + 2 * BOX;     // the parts of v'
    static constexpr int OFF_SNAP = OFF_VP + PARTS * BOX;  // D rows x 64 columns
    static constexpr int OFF_G = OFF_SNAP + D * 128;   // gate sums, two blocks
    static constexpr int OFF_MISC = OFF_G + 1024;
    static constexpr int SMEM_BYTES = 1024 + OFF_MISC + 512;
    // (two CTAs of one SM would wait for TMEM, of which each takes all 512 columns)
    static_assert(SMEM_BYTES > 114 * 1024 && SMEM_BYTES <= 227 * 1024, "one CTA per SM");
    // TMEM: two scores buffers, of which P takes the first 64 columns; q S; P v; k^T v', of the
    // first part and of the other two
    static constexpr int TM_S = 0, TM_QS = 256, TM_PV = 320, TM_KV = 384;
    static constexpr int GROUP = 128, THREADS = 6 * GROUP;
    // registers a thread: launched with 80; the shares of the six warpgroups add up to 6 * 80
    static constexpr int R_LAUNCH = 80, R_MISC = 40, R_KV = 144, R_P = 80, R_O = 88, R_V = 64;
    static_assert(R_MISC + R_KV + R_P + R_O + 2 * R_V == 6 * R_LAUNCH, "register shares");
    static constexpr uint32_t ID_S = idesc_bf16_f32(128, 128, 0, 0);
    static constexpr uint32_t ID_O = idesc_bf16_f32(128, 64, 0, 1);
    static constexpr uint32_t ID_KV2 = idesc_bf16_f32(D, 128, 1, 1), ID_KV1 = idesc_bf16_f32(D, 64, 1, 1);
};

struct GatedPrefillMisc {
    uint64_t full_q[2], full_k[2], full_v[2];
    uint64_t empty_q[2];   // the scores and q S have read the slot
    uint64_t empty_k[2];   // the scores and k^T v'
    uint64_t empty_v[2];   // P v and group V; then group O, whose output passes through the slot
    uint64_t s_full[2], p_ready[2], o_free[2];
    uint64_t v_ready[4];   // a quarter of v' (32 tokens) written, its tail zeroed
    uint64_t v_free[4];    // its products are done
    uint64_t v_split[2];   // group V has read a block's values
    uint64_t tail_zeroed;  // single phase: rows behind the sequence's end, for P v
    uint64_t kv_full, kv_free;
    uint64_t snap_ready, qs_done;
    uint64_t o_full;
    uint64_t gates_ready[2], gates_free[2];
    uint64_t done;
    float sum[2];          // log-decay of a block, times log2(e)
    uint32_t tmem_base;
    int abort_flag;
};

// 16 consecutive TMEM columns of this thread's lane, from registers.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

template <int D>
__global__ void __launch_bounds__(GatedPrefillCfg<D>::THREADS, 1)
    gated_prefill_tc_kernel(const __grid_constant__ GatedPrefillParams p) {
    using C = GatedPrefillCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    GatedPrefillMisc *m = reinterpret_cast<GatedPrefillMisc *>(smem + C::OFF_MISC);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int vs = blockIdx.x % C::NVS;
    const int h = (blockIdx.x / C::NVS) % p.H, sg = blockIdx.x / (C::NVS * p.H);
    int rank, s, start, len, sid;
    p.tab.seg(sg, rank, s);
    p.tab.seqs.get(rank, start, len, sid);
    const int all = (len + C::C - 1) / C::C;
    const int b0 = s * p.tab.seg_blocks, nb = max(0, min(all, b0 + p.tab.seg_blocks) - b0);
    const int first_row = start + b0 * C::C, rows = min(len - b0 * C::C, nb * C::C);
    const uint64_t tlimit = p.timeout_ns;
    volatile int *abort_flag = &m->abort_flag;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m->full_q[i], 1);
            mbar_init(&m->full_k[i], 1);
            mbar_init(&m->full_v[i], 1);
            mbar_init(&m->empty_q[i], 2);
            mbar_init(&m->empty_k[i], 2);
            mbar_init(&m->empty_v[i], 4);
            mbar_init(&m->s_full[i], 1);
            mbar_init(&m->p_ready[i], C::GROUP);
            mbar_init(&m->o_free[i], C::GROUP);
            mbar_init(&m->v_split[i], 8);
            mbar_init(&m->gates_ready[i], 32);
            mbar_init(&m->gates_free[i], 20);  // the warps of groups KV, P, O and V
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&m->v_ready[i], 64);
            mbar_init(&m->v_free[i], 1);
        }
        mbar_init(&m->tail_zeroed, 2 * C::GROUP);
        mbar_init(&m->kv_full, 1);
        mbar_init(&m->kv_free, C::GROUP);
        mbar_init(&m->snap_ready, C::GROUP);
        mbar_init(&m->qs_done, 1);
        mbar_init(&m->o_full, 1);
        mbar_init(&m->done, 3);
        m->abort_flag = 0;
        fence_mbarrier_init_cluster();
        tma_prefetch_desc(&p.tmap_q);
        tma_prefetch_desc(&p.tmap_k);
        tma_prefetch_desc(&p.tmap_v);
        tma_prefetch_desc(&p.tmap_o);
    }
    if (warp == 1) {
        tmem_alloc(&m->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = m->tmem_base;
    previous_done();
    auto fail = [&]() {
        *abort_flag = 1;
        record_fault(DEV_TIMEOUT);
    };
    auto wwait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return warp_wait(bar, parity, abort_flag, tlimit);
    };
    // Parity of block b's phase of a barrier with two slots, and of one with a single slot.
    auto two = [](int b) { return (uint32_t)((b >> 1) & 1); };
    auto one = [](int b) { return (uint32_t)(b & 1); };
    auto q_at = [&](int b) { return sbase + C::OFF_Q + (uint32_t)((b & 1) * C::TILE); };
    auto k_at = [&](int b) { return sbase + C::OFF_K + (uint32_t)((b & 1) * C::TILE); };
    auto v_at = [&](int b) { return sbase + C::OFF_V + (uint32_t)((b & 1) * C::BOX); };
    auto gates_of = [&](int b, uint32_t (&x)[4]) {
        fetch_gates4(x, p.g, first_row + b * C::C, min(C::C, rows - b * C::C), p.H, h);
    };
    // the gate sums of block b, in shared memory (store_gate_sums); a warp that has read them
    // says so, and gates_ready of b + 2 needs that of every warp
    auto sums_of = [&](int b) { return reinterpret_cast<float *>(smem + C::OFF_G) + C::C * (b & 1); };
    auto gates_read = [&](int b) {
        reads_done();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m->gates_free[b & 1]);
    };
    const int group = warp >> 2, q = warp & 3;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    const int row = 32 * q + lane;  // this thread's row of a block in groups P and O

    // Every wait on a phase of a barrier below is exact: the next phase needs, through the
    // chain named beside it, that this wait has returned.
    if (group == 0) {
        reg_dec<C::R_MISC>();
        if (warp == 0) {
            // ------------------------------------------------------------ gate sums, TMA loads
            // The tiles of a block first: the gate sums wait for the last readers of the sums of
            // two blocks before.
            int nk = 0, nq = 0, nv = 0, done = 0;
            uint32_t raw[4];
            float gate[4];
            if (nb > 0) gates_of(0, raw);
            for (int b = 0; b < nb; ++b) {
                const int y = first_row + b * C::C, col = h * D;
                if (!wwait(&m->empty_k[b & 1], two(b) ^ 1u)) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&m->full_k[b & 1], (uint32_t)C::TILE);
                    for (int d = 0; d < C::DB; ++d)
                        tma_load_2d(k_at(b) + d * C::BOX, &p.tmap_k, col + 64 * d, y, &m->full_k[b & 1]);
                }
                ++nk;
                if (!wwait(&m->empty_q[b & 1], two(b) ^ 1u)) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&m->full_q[b & 1], (uint32_t)C::TILE);
                    for (int d = 0; d < C::DB; ++d)
                        tma_load_2d(q_at(b) + d * C::BOX, &p.tmap_q, col + 64 * d, y, &m->full_q[b & 1]);
                }
                ++nq;
                if (!wwait(&m->empty_v[b & 1], two(b) ^ 1u)) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&m->full_v[b & 1], (uint32_t)C::BOX);
                    tma_load_2d(v_at(b), &p.tmap_v, col + 64 * vs, y, &m->full_v[b & 1]);
                }
                ++nv;
                if (!wwait(&m->gates_free[b & 1], two(b) ^ 1u)) break;
                widen_gates4(gate, raw);
                store_gate_sums(sums_of(b), &m->sum[b & 1], gate);
                mbar_arrive(&m->gates_ready[b & 1]);
                if (b + 1 < nb) gates_of(b + 1, raw);
                ++done;
            }
            if (done < nb) fail();
            // loads that are still in flight land before the CTA ends
            for (int b = max(0, nk - 2); b < nk; ++b) mbar_wait(&m->full_k[b & 1], two(b), nullptr, tlimit);
            for (int b = max(0, nq - 2); b < nq; ++b) mbar_wait(&m->full_q[b & 1], two(b), nullptr, tlimit);
            for (int b = max(0, nv - 2); b < nv; ++b) mbar_wait(&m->full_v[b & 1], two(b), nullptr, tlimit);
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------------------------ scores
            const uint32_t leader = elect_leader();
            bool ok = true;
            for (int b = 0; b < nb; ++b) {
                // full_k, full_q: the slots' next loads need the commits below.  o_free of b - 2: P_{b-2},
                // in this buffer, has been read by its product; its next phase but one (block b) needs
                // these scores.
                if (!wwait(&m->full_k[b & 1], two(b)) || !wwait(&m->full_q[b & 1], two(b)) ||
                    (b >= 2 && !wwait(&m->o_free[b & 1], two(b - 2)))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t qd = desc_kmajor_sw128(q_at(b)), kd = desc_kmajor_sw128(k_at(b));
#pragma unroll 2
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t off = (uint32_t)((ks >> 2) * C::BOX + (ks & 3) * 32);
                    warp_mma_ss(leader, tmem + C::TM_S + 128 * (b & 1), desc_add(qd, off), desc_add(kd, off), C::ID_S,
                                ks > 0 ? 1u : 0u);
                }
                warp_commit(leader, &m->s_full[b & 1]);
                warp_commit(leader, &m->empty_q[b & 1]);
                warp_commit(leader, &m->empty_k[b & 1]);
            }
            if (!ok) fail();
            warp_commit(leader, &m->done);  // every issued MMA has finished before TMEM is freed
            mbar_wait(&m->done, 0u, nullptr, tlimit);
            __syncwarp();
        } else if (warp == 2) {
            // ------------------------------------------------------------ q S, P v
            const uint32_t leader = elect_leader();
            bool ok = true;
            for (int b = 0; b < nb; ++b) {
                // full_q, full_v: the slots' next loads need the commits below; p_ready of b + 2 needs
                // o_free of b, that these products; snap_ready of b + 1 needs qs_done of b; o_free of
                // b - 1 (both accumulators have been read): its next phase (b + 1) needs o_full of b + 1
                if (!wwait(&m->full_q[b & 1], two(b)) || !wwait(&m->snap_ready, one(b)) ||
                    (b >= 1 && !wwait(&m->o_free[(b - 1) & 1], two(b - 1)))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t qd = desc_kmajor_sw128(q_at(b)), sd = desc_mnmajor_sw128(sbase + C::OFF_SNAP, C::BOX);
#pragma unroll 2
                for (int ks = 0; ks < D / 16; ++ks)
                    warp_mma_ss(leader, tmem + C::TM_QS, desc_add(qd, (uint32_t)((ks >> 2) * C::BOX + (ks & 3) * 32)),
                                desc_add(sd, ks * 2048), C::ID_O, ks > 0 ? 1u : 0u);
                warp_commit(leader, &m->qs_done);
                warp_commit(leader, &m->empty_q[b & 1]);
                if (!wwait(&m->full_v[b & 1], two(b)) || !wwait(&m->p_ready[b & 1], two(b)) ||
                    (rows < (b + 1) * C::C && !wwait(&m->tail_zeroed, 0u))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t vd = desc_mnmajor_sw128(v_at(b), C::BOX);
#pragma unroll 2
                for (int ks = 0; ks < C::C / 16; ++ks)
                    warp_mma_ts(leader, tmem + C::TM_PV, tmem + C::TM_S + 128 * (b & 1) + 8 * ks,
                                desc_add(vd, ks * 2048), C::ID_O, ks > 0 ? 1u : 0u);
                warp_commit(leader, &m->o_full);
            }
            if (!ok) fail();
            warp_commit(leader, &m->done);
            mbar_wait(&m->done, 0u, nullptr, tlimit);
            __syncwarp();
        } else {
            // ------------------------------------------------------------ k^T v'
            const uint32_t leader = elect_leader();
            bool ok = true;
            for (int b = 0; ok && b < nb; ++b) {
                // full_k's next load needs the commit below; kv_free of b needs this product
                ok = wwait(&m->full_k[b & 1], two(b)) && (b < 1 || wwait(&m->kv_free, one(b - 1)));
                const uint64_t kd = desc_mnmajor_sw128(k_at(b), C::BOX),
                               vd = desc_mnmajor_sw128(sbase + C::OFF_VP, C::BOX);
#pragma unroll 1
                for (int u = 0; u < 4; ++u) {  // a quarter at a time: group V refills one while the others multiply
                    // v_ready of b + 1 needs v_free of b
                    if (!ok || !(ok = wwait(&m->v_ready[u], one(b)))) break;
                    tc_fence_after();
#pragma unroll
                    for (int ks = 2 * u; ks < 2 * u + 2; ++ks)
                        warp_mma_ss(leader, tmem + C::TM_KV, desc_add(kd, ks * 2048), desc_add(vd, ks * 2048), C::ID_KV2,
                                    ks > 0 ? 1u : 0u);
#pragma unroll
                    for (int ks = 2 * u; ks < 2 * u + 2; ++ks)
                        warp_mma_ss(leader, tmem + C::TM_KV + 64, desc_add(kd, ks * 2048),
                                    desc_add(vd, 2 * C::BOX + ks * 2048), C::ID_KV1, 1u);
                    warp_commit(leader, &m->v_free[u]);
                }
                if (ok) {
                    warp_commit(leader, &m->kv_full);
                    warp_commit(leader, &m->empty_k[b & 1]);
                }
            }
            if (!ok) fail();
            warp_commit(leader, &m->done);
            mbar_wait(&m->done, 0u, nullptr, tlimit);
            __syncwarp();
        }
    } else if (group == 1) {
        // ---------------------------------------------------------------- group KV: the state
        reg_inc<C::R_KV>();
        const int i = D == 128 ? 32 * q + lane : 16 * q + lane;  // state row (M = 64: see gated_state_tc.cuh)
        const bool i_ok = D == 128 || lane < 16;
        float X[64];
#pragma unroll
        for (int x = 0; x < 64; ++x) X[x] = 0.f;
        const float *from = nullptr;
        if (p.seg_in != nullptr)
            from = p.seg_in + ((size_t)sg * p.H + h) * D * D;
        else if (p.initial != nullptr)
            from = p.initial + ((size_t)sid * p.H + h) * D * D;
        if (from != nullptr && i_ok) {
            const float4 *src = reinterpret_cast<const float4 *>(from + (size_t)i * D + 64 * vs);
#pragma unroll
            for (int x = 0; x < 16; ++x) {
                const float4 f = src[x];
                X[4 * x] = f.x, X[4 * x + 1] = f.y, X[4 * x + 2] = f.z, X[4 * x + 3] = f.w;
            }
        }
        auto snapshot = [&]() {
            if (i_ok) {
                const uint32_t at = sbase + C::OFF_SNAP + i * 128;
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    st_shared_v4(at + ((x ^ (i & 7)) << 4), pack_bf16x2(X[8 * x], X[8 * x + 1]),
                                 pack_bf16x2(X[8 * x + 2], X[8 * x + 3]), pack_bf16x2(X[8 * x + 4], X[8 * x + 5]),
                                 pack_bf16x2(X[8 * x + 6], X[8 * x + 7]));
            }
            fence_proxy_async_smem();
            mbar_arrive(&m->snap_ready);
        };
        if (nb > 0) snapshot();
        bool ok = true;
        for (int b = 0; b < nb; ++b) {
            if (!wwait(&m->gates_ready[b & 1], two(b))) {
                ok = false;
                break;
            }
            const float decay = exp2f(m->sum[b & 1]);
            gates_read(b);
            // kv_full of b + 1 needs kv_free of b
            if (!wwait(&m->kv_full, one(b))) {
                ok = false;
                break;
            }
            tc_fence_after();
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t a[32], c[32];
                tmem_ld32(tmem + C::TM_KV + 64 + 32 * half + lanes, c);
                tmem_ld32(tmem + C::TM_KV + 32 * half + lanes, a);
                tmem_ld_wait();
                if (half == 1) {
                    tc_fence_before();
                    mbar_arrive(&m->kv_free);
                }
#pragma unroll
                for (int x = 0; x < 32; ++x)
                    X[32 * half + x] = fmaf(decay, X[32 * half + x], __uint_as_float(a[x]) + __uint_as_float(c[x]));
            }
            if (b + 1 < nb) {
                // qs_done of b + 1 needs the snapshot below
                if (!wwait(&m->qs_done, one(b))) {
                    ok = false;
                    break;
                }
                snapshot();
            }
        }
        if (ok && p.fin != nullptr && s == p.tab.num_segs(rank) - 1 && i_ok) {
            float4 *d4 = reinterpret_cast<float4 *>(p.fin + (((size_t)sid * p.H + h) * D + i) * D + 64 * vs);
#pragma unroll
            for (int x = 0; x < 16; ++x) d4[x] = make_float4(X[4 * x], X[4 * x + 1], X[4 * x + 2], X[4 * x + 3]);
        }
        if (!ok) fail();
    } else if (group == 2) {
        // ---------------------------------------------------------------- group P
        bool ok = true;
        for (int b = 0; b < nb; ++b) {
            const float *sG = sums_of(b);
            // s_full of b + 2 needs o_free of b
            if (!wwait(&m->gates_ready[b & 1], two(b)) || !wwait(&m->s_full[b & 1], two(b))) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t si = __float_as_uint(sG[row]);
            const uint64_t s2 = pair_f32(si, si);
            const uint32_t tS = tmem + C::TM_S + 128 * (b & 1) + lanes;
            // columns 32 cc .. of the scores become columns 16 cc .. of P, over scores that this
            // lane has read
            auto decayed = [&](int cc, const uint32_t (&sc)[32], uint32_t (&w)[16]) {
#pragma unroll
                for (int y = 0; y < 32; y += 4) {
                    const ulonglong2 sj = *reinterpret_cast<const ulonglong2 *>(&sG[32 * cc + y]);
                    w[y / 2] = pack_f32x2(mul_f32x2(pair_f32(sc[y], sc[y + 1]), ex2_f32x2(sub_f32x2(sj.x, s2))));
                    w[y / 2 + 1] =
                        pack_f32x2(mul_f32x2(pair_f32(sc[y + 2], sc[y + 3]), ex2_f32x2(sub_f32x2(sj.y, s2))));
                }
            };
#pragma unroll 1
            for (int cc = 0; cc < 4; ++cc) {
                uint32_t w[16];
                if (cc <= q) {
                    uint32_t sc[32];
                    tmem_ld32(tS + 32 * cc, sc);
                    tmem_ld_wait();
                    decayed(cc, sc, w);
                    if (cc == q) {  // columns behind this row, whatever they hold, give 0
#pragma unroll
                        for (int y = 0; y < 16; ++y)
                            w[y] &= 2 * y + 1 <= lane ? 0xffffffffu : 2 * y <= lane ? 0x0000ffffu : 0u;
                    }
                } else {
#pragma unroll
                    for (int y = 0; y < 16; ++y) w[y] = 0u;
                }
                tmem_st16(tS + 16 * cc, w);
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&m->p_ready[b & 1]);
            gates_read(b);
        }
        if (!ok) fail();
    } else if (group == 3) {
        // ---------------------------------------------------------------- group O
        reg_inc<C::R_O>();
        bool ok = true;
        for (int b = 0; b < nb; ++b) {
            if (!wwait(&m->gates_ready[b & 1], two(b))) {
                ok = false;
                break;
            }
            const float w = ex2(m->sum[b & 1] - sums_of(b)[row]);
            gates_read(b);
            // o_full of b + 1 needs o_free of b
            if (!wwait(&m->o_full, one(b))) {
                ok = false;
                break;
            }
            tc_fence_after();
            // The values' slot takes the output on its way: P v has read it (o_full), group V too
            // (v_split, below), and each warp stages and stores its own 32 rows.  Stores from
            // registers would touch 32 rows each: 32 passes of the memory pipe per 16 bytes of a row.
            if (!wwait(&m->v_split[b & 1], two(b))) {  // that of b + 2 needs this block's empty_v
                ok = false;
                break;
            }
            const uint32_t stage = v_at(b) + 32 * q * 128;
#pragma unroll 1
            for (int x = 0; x < 4; ++x) {
                uint32_t a[16], c[16];
                tmem_ld16(tmem + C::TM_QS + 16 * x + lanes, a);
                tmem_ld16(tmem + C::TM_PV + 16 * x + lanes, c);
                tmem_ld_wait();
                float y[16];
#pragma unroll
                for (int z = 0; z < 16; ++z) y[z] = fmaf(w, __uint_as_float(a[z]), __uint_as_float(c[z]));
#pragma unroll
                for (int z = 0; z < 2; ++z)
                    st_shared_u4(stage + lane * 128 + (((2 * x + z) ^ (lane & 7)) << 4), pack_chunk(&y[8 * z]));
            }
            tc_fence_before();
            mbar_arrive(&m->o_free[b & 1]);
            const int r0 = b * C::C + 32 * q;
            if (r0 + 32 <= rows) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_2d(&p.tmap_o, stage, h * D + 64 * vs, first_row + r0);
                    bulk_commit_group();
                    bulk_wait_read_all();
                }
            } else if (r0 + lane < rows) {  // the sequence's last rows, one lane each
                uint4 *dst = reinterpret_cast<uint4 *>(p.o + ((size_t)(first_row + r0 + lane) * p.H + h) * D + 64 * vs);
#pragma unroll 1
                for (int z = 0; z < 8; ++z) dst[z] = ld_shared_v4(stage + lane * 128 + ((z ^ (lane & 7)) << 4));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&m->empty_v[b & 1]);
        }
        if (lane == 0) bulk_wait_all();
        if (!ok) fail();
    } else {
        // ---------------------------------------------------------------- groups V: 16 rows a warp
        reg_dec<C::R_V>();
        const int w8 = warp - 16, u = w8 >> 1;  // this warp's sixteenth rows lie in quarter u
        bool ok = true;
        for (int b = 0; b < nb; ++b) {
            const int nv = min(C::C, rows - b * C::C);
            // full_v's next load needs the arrival below; v_free of b needs v_ready of b
            if (!wwait(&m->gates_ready[b & 1], two(b)) || !wwait(&m->full_v[b & 1], two(b)) ||
                (b >= 1 && !wwait(&m->v_free[u], one(b - 1)))) {
                ok = false;
                break;
            }
            if (nv < C::C) {
                // the last block: rows of the next sequence must not enter P v or k^T v' (the
                // scores mask them); 0 times what they hold could be a NaN
                if (!wwait(&m->full_k[b & 1], two(b))) {
                    ok = false;
                    break;
                }
                for (int c = max(nv, 16 * w8) * 8 + lane; c < (16 * w8 + 16) * 8; c += 32) {
                    st_shared_v4(v_at(b) + c * 16, 0u, 0u, 0u, 0u);
                    for (int d = 0; d < C::DB; ++d) st_shared_v4(k_at(b) + d * C::BOX + c * 16, 0u, 0u, 0u, 0u);
                }
                __syncwarp();
                fence_proxy_async_smem();
                mbar_arrive(&m->tail_zeroed);
            }
#pragma unroll 1
            for (int x = 0; x < 4; ++x) {
                const int c = w8 * 128 + x * 32 + lane, r = c >> 3;
                uint4 part[C::PARTS];
                split_chunk(ld_shared_v4(v_at(b) + c * 16), exp2f(sums_of(b)[r]), r < nv, part);
#pragma unroll
                for (int y = 0; y < C::PARTS; ++y) st_shared_u4(sbase + C::OFF_VP + y * C::BOX + c * 16, part[y]);
            }
            fence_proxy_async_smem();
            mbar_arrive(&m->v_ready[u]);
            gates_read(b);
            if (lane == 0) mbar_arrive(&m->v_split[b & 1]);
        }
        if (!ok) fail();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace la
