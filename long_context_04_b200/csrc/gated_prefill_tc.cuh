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
// three bf16 parts (see gated_state_tc.cuh) in two accumulators, [part 0 | parts 1 + 2].
// P goes back to TMEM over the scores it came from and is read there as the left factor.
//
// Warpgroups (640 threads; registers are moved to the group that holds the state):
//   0  warp 0 TMA loads; warp 1 issues the scores and k^T v'; warp 2 issues q S and P v
//   1  group KV: the fp32 state in registers, its bf16 snapshot for q S, the final state
//   2  group P: scores -> decay, mask -> P
//   3  group O: e^{G_i} (q S) + P v -> bf16 -> global
//   4  group V: v -> v', zeros behind the sequence's end
// q, k and v have rings of two slots each, released by their last readers, so that the next
// block's scores and k^T v' run while this block's output is still being formed.
//
// Limits per block and CTA at D = 128: HBM 64 KB of a pair's 128 KB (2360 cycles of the
// measured copy rate over 128 CTAs), tensor 1900 cycles, shared memory about 2900 cycles
// (tiles in, operands out, v' written and read).
#pragma once

#include "gated_state_tc.cuh"

namespace la {

struct GatedPrefillParams {
    CUtensorMap tmap_q, tmap_k, tmap_v;   // [T][H*D], box 64 x 128
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
    static constexpr int NVS = D / 64;
    static constexpr int DB = D / 64;
    static constexpr int BOX = C * 128;
    static constexpr int TILE = DB * BOX;              // q or k
    static constexpr int OFF_Q = 0, OFF_K = 2 * TILE, OFF_V = 4 * TILE;
    static constexpr int OFF_VP = OFF_V + 2 * BOX;     // three parts of v'
    static constexpr int OFF_SNAP = OFF_VP + 3 * BOX;  // D rows x 64 columns
    static constexpr int OFF_W = OFF_SNAP + D * 128;   // decays of v's rows
    static constexpr int OFF_G = OFF_W + 512;          // 2 x 128 sums of log-decays (times log2 e)
    static constexpr int OFF_MISC = OFF_G + 1024;
    static constexpr int SMEM_USED = 1024 + OFF_MISC + 512;
    // above half of the SM's shared memory: two CTAs of one SM would wait for TMEM
    static constexpr int SMEM_BYTES = SMEM_USED < 120 * 1024 ? 120 * 1024 : SMEM_USED;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
    static constexpr int TM_S = 0, TM_QS = 256, TM_PV = 320, TM_KV = 384;
    static constexpr int GROUP = 128, THREADS = 5 * GROUP;
    // registers a thread: launched with 96; the five shares add up to 5 * 96
    static constexpr int R_MISC = 40, R_KV = 152, R_P = 104, R_O = 96, R_V = 88;
    static_assert(R_MISC + R_KV + R_P + R_O + R_V == 5 * 96, "register shares");
    static constexpr uint32_t ID_S = idesc_bf16_f32(128, 128, 0, 0);
    static constexpr uint32_t ID_O = idesc_bf16_f32(128, 64, 0, 1);
    static constexpr uint32_t ID_KV2 = idesc_bf16_f32(D, 128, 1, 1);
    static constexpr uint32_t ID_KV1 = idesc_bf16_f32(D, 64, 1, 1);
};

struct GatedPrefillMisc {
    uint64_t full_q[2], full_k[2], full_v[2];
    uint64_t empty_q[2];   // the scores and q S have read the slot
    uint64_t empty_k[2];   // the scores and k^T v'
    uint64_t empty_v[2];   // P v and group V
    uint64_t s_full[2], p_ready[2], pv_done[2];
    uint64_t v_ready;      // v' written (and the tail zeroed)
    uint64_t tail_zeroed;  // single phase: rows behind the sequence's end, for P v
    uint64_t kv_full, kv_free;
    uint64_t snap_ready, qs_done;
    uint64_t o_full, o_free;
    uint64_t done;
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
            mbar_init(&m->empty_k[i], 1);
            mbar_init(&m->empty_v[i], 1 + C::GROUP);
            mbar_init(&m->s_full[i], 1);
            mbar_init(&m->p_ready[i], C::GROUP);
            mbar_init(&m->pv_done[i], 1);
        }
        mbar_init(&m->v_ready, C::GROUP);
        mbar_init(&m->tail_zeroed, C::GROUP);
        mbar_init(&m->kv_full, 1);
        mbar_init(&m->kv_free, C::GROUP);
        mbar_init(&m->snap_ready, C::GROUP);
        mbar_init(&m->qs_done, 1);
        mbar_init(&m->o_full, 1);
        mbar_init(&m->o_free, C::GROUP);
        mbar_init(&m->done, 2);
        m->abort_flag = 0;
        fence_mbarrier_init_cluster();
        tma_prefetch_desc(&p.tmap_q);
        tma_prefetch_desc(&p.tmap_k);
        tma_prefetch_desc(&p.tmap_v);
    }
    if (warp == 1) {
        tmem_alloc(&m->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = m->tmem_base;
    auto fail = [&]() {
        *abort_flag = 1;
        record_fault(DEV_TIMEOUT);
    };
    auto wwait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, tlimit)) != 0;
    };
    // Parity of block b's phase of a barrier with two slots, and of one with a single slot.
    auto two = [](int b) { return (uint32_t)((b >> 1) & 1); };
    auto one = [](int b) { return (uint32_t)(b & 1); };
    auto q_at = [&](int b) { return sbase + C::OFF_Q + (uint32_t)((b & 1) * C::TILE); };
    auto k_at = [&](int b) { return sbase + C::OFF_K + (uint32_t)((b & 1) * C::TILE); };
    auto v_at = [&](int b) { return sbase + C::OFF_V + (uint32_t)((b & 1) * C::BOX); };
    auto gates_of = [&](int b, float (&x)[4]) {
        load_gates4(x, p.g, first_row + b * C::C, min(C::C, rows - b * C::C), p.H, h);
    };
    const int group = warp >> 2, q = warp & 3;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    const int row = 32 * q + lane;  // this thread's row of a block in groups P and O

    // Every wait on a phase of a barrier below is exact: the next phase needs, through the
    // chain named beside it, that this wait has returned.
    if (group == 0) {
        reg_dec<C::R_MISC>();
        if (warp == 0) {
            // ------------------------------------------------------------ TMA loads
            if (lane == 0) {
                int nk = 0, nq = 0, nv = 0;
                for (int b = 0; b < nb; ++b) {
                    const int y = first_row + b * C::C, col = h * D;
                    if (!mbar_wait(&m->empty_k[b & 1], two(b) ^ 1u, abort_flag, tlimit)) break;
                    mbar_arrive_expect_tx(&m->full_k[b & 1], (uint32_t)C::TILE);
                    for (int d = 0; d < C::DB; ++d)
                        tma_load_2d(k_at(b) + d * C::BOX, &p.tmap_k, col + 64 * d, y, &m->full_k[b & 1]);
                    ++nk;
                    if (!mbar_wait(&m->empty_q[b & 1], two(b) ^ 1u, abort_flag, tlimit)) break;
                    mbar_arrive_expect_tx(&m->full_q[b & 1], (uint32_t)C::TILE);
                    for (int d = 0; d < C::DB; ++d)
                        tma_load_2d(q_at(b) + d * C::BOX, &p.tmap_q, col + 64 * d, y, &m->full_q[b & 1]);
                    ++nq;
                    if (!mbar_wait(&m->empty_v[b & 1], two(b) ^ 1u, abort_flag, tlimit)) break;
                    mbar_arrive_expect_tx(&m->full_v[b & 1], (uint32_t)C::BOX);
                    tma_load_2d(v_at(b), &p.tmap_v, col + 64 * vs, y, &m->full_v[b & 1]);
                    ++nv;
                }
                if (nv < nb) fail();
                // loads that are still in flight land before the CTA ends
                for (int b = max(0, nk - 2); b < nk; ++b) mbar_wait(&m->full_k[b & 1], two(b), nullptr, tlimit);
                for (int b = max(0, nq - 2); b < nq; ++b) mbar_wait(&m->full_q[b & 1], two(b), nullptr, tlimit);
                for (int b = max(0, nv - 2); b < nv; ++b) mbar_wait(&m->full_v[b & 1], two(b), nullptr, tlimit);
            }
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------------------------ scores, k^T v'
            bool ok = true;
            for (int b = 0; ok && b < nb; ++b) {
                // full_k, full_q: the slots' next loads need this warp's commits of block b.
                // pv_done of b - 2: P_{b-2}, in this scores buffer, has been read; its next phase
                // (block b) needs the scores of b.
                if (!wwait(&m->full_k[b & 1], two(b)) || !wwait(&m->full_q[b & 1], two(b)) ||
                    (b >= 2 && !wwait(&m->pv_done[b & 1], two(b - 2)))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (lane == 0) {
                    const uint64_t qd = desc_kmajor_sw128(q_at(b)), kd = desc_kmajor_sw128(k_at(b));
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t off = (uint32_t)((ks >> 2) * C::BOX + (ks & 3) * 32);
                        mma_bf16_ss(tmem + C::TM_S + 128 * (b & 1), desc_add(qd, off), desc_add(kd, off), C::ID_S,
                                    ks > 0 ? 1u : 0u);
                    }
                    mma_commit(&m->s_full[b & 1]);
                    mma_commit(&m->empty_q[b & 1]);
                }
                __syncwarp();
                // v_ready of b + 1 needs this product; kv_free of b needs it too
                if (!wwait(&m->v_ready, one(b)) || (b >= 1 && !wwait(&m->kv_free, one(b - 1)))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (lane == 0) {
                    const uint64_t kd = desc_mnmajor_sw128(k_at(b), C::BOX),
                                   vd = desc_mnmajor_sw128(sbase + C::OFF_VP, C::BOX);
#pragma unroll
                    for (int ks = 0; ks < C::C / 16; ++ks)
                        mma_bf16_ss(tmem + C::TM_KV, desc_add(kd, ks * 2048), desc_add(vd, ks * 2048), C::ID_KV2,
                                    ks > 0 ? 1u : 0u);
#pragma unroll
                    for (int ks = 0; ks < C::C / 16; ++ks)
                        mma_bf16_ss(tmem + C::TM_KV + 64, desc_add(kd, ks * 2048),
                                    desc_add(vd, 2 * C::BOX + ks * 2048), C::ID_KV1, 1u);
                    mma_commit(&m->kv_full);
                    mma_commit(&m->empty_k[b & 1]);
                }
                __syncwarp();
            }
            if (!ok) fail();
            if (lane == 0) {  // every issued MMA has finished before TMEM is freed
                mma_commit(&m->done);
                mbar_wait(&m->done, 0u, nullptr, tlimit);
            }
            __syncwarp();
        } else if (warp == 2) {
            // ------------------------------------------------------------ q S, P v
            bool ok = true;
            for (int b = 0; ok && b < nb; ++b) {
                // snap_ready of b + 1 needs qs_done of b; o_free of b needs o_full of b;
                // full_q's next load needs the commit below
                if (!wwait(&m->full_q[b & 1], two(b)) || !wwait(&m->snap_ready, one(b)) ||
                    (b >= 1 && !wwait(&m->o_free, one(b - 1)))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (lane == 0) {
                    const uint64_t qd = desc_kmajor_sw128(q_at(b)),
                                   sd = desc_mnmajor_sw128(sbase + C::OFF_SNAP, C::BOX);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        mma_bf16_ss(tmem + C::TM_QS, desc_add(qd, (uint32_t)((ks >> 2) * C::BOX + (ks & 3) * 32)),
                                    desc_add(sd, ks * 2048), C::ID_O, ks > 0 ? 1u : 0u);
                    mma_commit(&m->qs_done);
                    mma_commit(&m->empty_q[b & 1]);
                }
                __syncwarp();
                // full_v's next load and p_ready of b + 2 need this product
                if (!wwait(&m->full_v[b & 1], two(b)) || !wwait(&m->p_ready[b & 1], two(b)) ||
                    (rows < (b + 1) * C::C && !wwait(&m->tail_zeroed, 0u))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (lane == 0) {
                    const uint64_t vd = desc_mnmajor_sw128(v_at(b), C::BOX);
#pragma unroll
                    for (int ks = 0; ks < C::C / 16; ++ks)
                        mma_bf16_ts(tmem + C::TM_PV, tmem + C::TM_S + 128 * (b & 1) + 8 * ks,
                                    desc_add(vd, ks * 2048), C::ID_O, ks > 0 ? 1u : 0u);
                    mma_commit(&m->o_full);
                    mma_commit(&m->pv_done[b & 1]);
                    mma_commit(&m->empty_v[b & 1]);
                }
                __syncwarp();
            }
            if (!ok) fail();
            if (lane == 0) {
                mma_commit(&m->done);
                mbar_wait(&m->done, 0u, nullptr, tlimit);
            }
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
        float gate[4];
        if (nb > 0) {
            gates_of(0, gate);
            snapshot();
        }
        bool ok = true;
        for (int b = 0; b < nb; ++b) {
            float G = (gate[0] + gate[1]) + (gate[2] + gate[3]);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) G += __shfl_xor_sync(0xffffffffu, G, off);
            const float decay = expf(G);
            if (b + 1 < nb) gates_of(b + 1, gate);
            // kv_full of b + 1 needs kv_free of b
            if (!wwait(&m->kv_full, one(b))) {
                ok = false;
                break;
            }
            tc_fence_after();
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t a[32], c[32];
                tmem_ld32(tmem + C::TM_KV + 32 * half + lanes, a);
                tmem_ld32(tmem + C::TM_KV + 64 + 32 * half + lanes, c);
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
        reg_inc<C::R_P>();
        float gate[4], sums[4];
        if (nb > 0) gates_of(0, gate);
        bool ok = true;
        for (int b = 0; b < nb; ++b) {
            // The group's four warps write equal values, each for its own reading.  Behind the wait
            // for s_full a warp is at most one block ahead of another (s_full of b + 2 needs P_b of
            // all), so two buffers suffice.
            float *sG = reinterpret_cast<float *>(smem + C::OFF_G) + 128 * (b & 1);
            prefix_gates4(gate, sums);
            if (b + 1 < nb) gates_of(b + 1, gate);
            // s_full of b + 2 needs pv_done of b
            if (!wwait(&m->s_full[b & 1], two(b))) {
                ok = false;
                break;
            }
            tc_fence_after();
            *reinterpret_cast<float4 *>(&sG[4 * lane]) =
                make_float4(sums[0] * 1.4426950408889634f, sums[1] * 1.4426950408889634f,
                            sums[2] * 1.4426950408889634f, sums[3] * 1.4426950408889634f);
            __syncwarp();
            const float Gi = sG[row];
            const uint32_t tS = tmem + C::TM_S + 128 * (b & 1) + lanes;
#pragma unroll 1
            for (int cc = 0; cc < 4; ++cc) {
                // columns 32 cc .. of the scores become columns 16 cc .. of P, over scores that
                // this lane has read
                uint32_t w[16];
                if (cc <= q) {
                    uint32_t sc[32];
                    tmem_ld32(tS + 32 * cc, sc);
                    tmem_ld_wait();
                    const int seen = cc < q ? 32 : lane + 1;
#pragma unroll
                    for (int y = 0; y < 32; y += 4) {
                        const float4 Gj = *reinterpret_cast<const float4 *>(&sG[32 * cc + y]);
                        const float p0 = y < seen ? __uint_as_float(sc[y]) * ex2(Gi - Gj.x) : 0.f;
                        const float p1 = y + 1 < seen ? __uint_as_float(sc[y + 1]) * ex2(Gi - Gj.y) : 0.f;
                        const float p2 = y + 2 < seen ? __uint_as_float(sc[y + 2]) * ex2(Gi - Gj.z) : 0.f;
                        const float p3 = y + 3 < seen ? __uint_as_float(sc[y + 3]) * ex2(Gi - Gj.w) : 0.f;
                        w[y / 2] = pack_bf16x2(p0, p1);
                        w[y / 2 + 1] = pack_bf16x2(p2, p3);
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
        }
        if (!ok) fail();
    } else if (group == 3) {
        // ---------------------------------------------------------------- group O
        float gate[4], sums[4];
        if (nb > 0) gates_of(0, gate);
        bool ok = true;
        for (int b = 0; b < nb; ++b) {
            prefix_gates4(gate, sums);
            if (b + 1 < nb) gates_of(b + 1, gate);
            // G of this thread's row: element lane % 4 of lane 8 q + lane / 4
            float G = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float y = __shfl_sync(0xffffffffu, sums[e], 8 * q + (lane >> 2));
                if ((lane & 3) == e) G = y;
            }
            const float w = expf(G);
            // o_full of b + 1 needs o_free of b
            if (!wwait(&m->o_full, one(b))) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint4 *dst = reinterpret_cast<uint4 *>(p.o + ((size_t)(first_row + b * C::C + row) * p.H + h) * D + 64 * vs);
            const bool mine = b * C::C + row < rows;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t a[32], c[32];
                tmem_ld32(tmem + C::TM_QS + 32 * half + lanes, a);
                tmem_ld32(tmem + C::TM_PV + 32 * half + lanes, c);
                tmem_ld_wait();
                if (half == 1) {
                    tc_fence_before();
                    mbar_arrive(&m->o_free);
                }
                float y[32];
#pragma unroll
                for (int x = 0; x < 32; ++x) y[x] = fmaf(w, __uint_as_float(a[x]), __uint_as_float(c[x]));
                if (mine) {
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        dst[4 * half + x] =
                            make_uint4(pack_bf16x2(y[8 * x], y[8 * x + 1]), pack_bf16x2(y[8 * x + 2], y[8 * x + 3]),
                                       pack_bf16x2(y[8 * x + 4], y[8 * x + 5]), pack_bf16x2(y[8 * x + 6], y[8 * x + 7]));
                }
            }
        }
        if (!ok) fail();
    } else {
        // ---------------------------------------------------------------- group V
        reg_dec<C::R_V>();
        float *sW = reinterpret_cast<float *>(smem + C::OFF_W);  // each warp its own 32 rows
        float gate[4], sums[4];
        if (nb > 0) gates_of(0, gate);
        bool ok = true;
        for (int b = 0; b < nb; ++b) {
            const int nv = min(C::C, rows - b * C::C);
            suffix_gates4(gate, sums);
            if (b + 1 < nb) gates_of(b + 1, gate);
            __syncwarp();
            if (lane >> 3 == q)
                *reinterpret_cast<float4 *>(&sW[4 * lane]) =
                    make_float4(expf(sums[0]), expf(sums[1]), expf(sums[2]), expf(sums[3]));
            __syncwarp();
            // full_v's next load needs the arrival below; kv_full of b - 1: v' of b - 1 has been
            // read, and kv_full of b needs v' of b
            if (!wwait(&m->full_v[b & 1], two(b)) || (b >= 1 && !wwait(&m->kv_full, one(b - 1)))) {
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
                for (int c = nv * 8 + (q * 32 + lane); c < C::C * 8; c += C::GROUP) {
                    st_shared_v4(v_at(b) + c * 16, 0u, 0u, 0u, 0u);
                    for (int d = 0; d < C::DB; ++d) st_shared_v4(k_at(b) + d * C::BOX + c * 16, 0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                mbar_arrive(&m->tail_zeroed);
            }
#pragma unroll 2
            for (int x = 0; x < 8; ++x) {
                const int c = q * 256 + x * 32 + lane, r = c >> 3;
                uint4 p0, p1, p2;
                split3(ld_shared_v4(v_at(b) + c * 16), sW[r], r < nv, p0, p1, p2);
                const uint32_t to = sbase + C::OFF_VP + c * 16;
                st_shared_u4(to, p0);
                st_shared_u4(to + C::BOX, p1);
                st_shared_u4(to + 2 * C::BOX, p2);
            }
            fence_proxy_async_smem();
            mbar_arrive(&m->v_ready);
            mbar_arrive(&m->empty_v[b & 1]);
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
