// Gradients of gated lightning attention on the tensor cores (bf16), one block of 128 tokens
// of one head at a time: from the state S at the block's start and the gradient dS of the state
// at its end (the state scans' snapshots, two bf16 parts each), every block stands alone.
//
//   scores   s = q k^T, t = do v^T;  P = s (.) decay,  dP = t (.) decay     (j <= i)
//   dq = e^{G_i} (do S^T)        + dP k
//   dk = e^{G_C - G_j} (v dS^T)  + dP^T q
//   dv = e^{G_C - G_j} (k dS)    + P^T do
//   dg as in gated.cuh, from W = dP (.) s and the row sums of q . dq and k . dk of the first
//   terms.
//
// The first terms of dq and dk, from whose rows dg's sums come, use both parts of S and dS; the
// first term of dv, a vector that no sum follows, the first part of dS alone.  P and dP are one
// bf16 number each, as operands of the last products; W is formed from the fp32 values.
//
// A persistent CTA per SM.  Shared memory (D = 128): q, k, v, do 32 KB each, the first parts of S
// and dS 32 KB each, a slot of 16 KB through which the second parts pass, 64 columns at a time; P
// takes the place of v and dP that of S once the products that read those are done.
// TMEM, 512 columns: s, t, dq, dk; the two terms of dv take the places of s and t.  The decays
// of the first terms differ by row: those of dq and dk are scaled in TMEM and the second
// products accumulate on top, the two of dv are added on the way out.  The products, in this
// order (lo: of a second part; D = 64 has both parts in place):
//   t, v dS^T, lo, s, do S^T, lo  ->  P, dP;  lo, lo  ->  scaling;  k dS; P^T do; dP k; dP^T q.
// P and dP are each stored once, [i][j]: as the left factor of dP k they are read along j, as
// the transposed left factor of the other two along i.
//
// Warps: 0 TMA loads and gate sums; 1 MMA issue; 2-9 (group A) scores -> P, dP, W, then dv and
// dk out; 10-13 (group B) scaling of the first terms and their row sums, then dq out; 14 dg.
// Every barrier completes one phase per block (the slot's as many as parts pass).  The next
// block's tiles are loaded as their places come free and multiplied (t, s and the first terms)
// while this one's results go out.  (Fetching them into L2 ahead cost 6 % of a call: the fetches
// came between the loads that a block waits for.)
//
// HBM: 14 D bytes of tiles and results and 8 D^2 / 128 bytes of snapshots per token and head
// (2816 at D = 128); tensor: 10 products of 512 cycles per block.  At 8192 tokens, 64 heads,
// D = 128: 291 us, 5.1 TB/s, tensor cores busy for 31 %; with one CTA per SM (shared memory
// and TMEM are full) the phases of a block that wait for one another bound it: without the second
// parts it took 242 us, and half of the difference is the wait for one load after the other.  A
// call of that size with its two scans takes 535 us.
#pragma once

#include "gated_state_tc.cuh"

namespace la {

struct GatedBackwardParams {
    CUtensorMap tmap_q, tmap_k, tmap_v, tmap_do;  // [T][H*D], box 64 x 128
    CUtensorMap tmap_s, tmap_ds;                  // [blocks * H][2 parts][D][D], box 64 x D
    const __nv_bfloat16 *g;
    const float *through;  // [blocks][H][8 D / 64] parts of e^{G_C} <dS, S>, or nullptr
    __nv_bfloat16 *dq, *dk, *dv, *dg;
    int H;
    int have_s, have_ds;   // snapshots of the state, of its gradient (else zero)
    unsigned long long timeout_ns;
    GatedTable tab;
};

template <int D>
struct GatedBackwardCfg {
    static constexpr int C = 128;
    static constexpr int DB = D / 64;
    static constexpr int BOX = C * 128;         // 64 columns x 128 rows
    static constexpr int SBOX = D * 128;        // 64 columns x D rows of a state
    static constexpr int TILE = DB * BOX;
    static constexpr int PT = 2 * BOX;          // P or dP
    static constexpr int OFF_Q = 0, OFF_K = TILE, OFF_DO = 2 * TILE, OFF_V = 3 * TILE;
    static constexpr int OFF_S = 4 * TILE, OFF_DS = OFF_S + PT;
    static constexpr int OFF_P = D == 128 ? OFF_V : OFF_DS + PT;  // D = 64: v is too small for P
    static constexpr int OFF_DP = OFF_S;
    // The second parts of S and dS.  D = 64: behind the first ones.  D = 128 (STREAM): a slot of
    // 64 columns, through which those of dS and then of S pass, LOWS in all.
    static constexpr bool STREAM = D == 128;
    static constexpr int OFF_LOW = OFF_S + 2 * PT + (D == 128 ? 0 : PT);
    static constexpr int OFF_STAGE = OFF_LOW + (STREAM ? SBOX : 0);         // 1 KB per storing warp
    static constexpr int OFF_F = OFF_STAGE + 12 * 1024;                     // 9 arrays of 128 floats
    static constexpr int OFF_MISC = OFF_F + 9 * 512;
    static constexpr int SMEM_BYTES = 1024 + OFF_MISC + 512;
    static_assert((STREAM ? DB : 2) * SBOX <= PT && (D != 128 || TILE == PT), "places of P and dP");
    static_assert(SMEM_BYTES > 114 * 1024 && SMEM_BYTES <= 227 * 1024, "one CTA per SM");
    static constexpr int TM_S = 0, TM_T = 128, TM_DQ = 256, TM_DK = 384, TM_DV1 = 0, TM_DV2 = 128;
    static constexpr int GROUP_A = 256, GROUP_B = 128, THREADS = 96 + GROUP_A + GROUP_B;
    static constexpr uint32_t ID_S = idesc_bf16_f32(128, 128, 0, 0);
    static constexpr uint32_t ID_KK = idesc_bf16_f32(128, D, 0, 0);
    static constexpr uint32_t ID_KN = idesc_bf16_f32(128, D, 0, 1);
    static constexpr uint32_t ID_NN = idesc_bf16_f32(128, D, 1, 1);
};

struct GatedBackwardMisc {
    uint64_t full_vo, full_k, full_qs, full_ds;  // v, do; k; q, S; dS landed
    uint64_t low_full, low_free;          // STREAM: 64 columns of a second part landed, multiplied
    uint64_t low_done;                    // STREAM: do S^T with S's second part too
    uint64_t gates;                       // gate sums of the block written
    uint64_t first_full;                  // s, t, do S^T (STREAM: of S's first part), v dS^T
    uint64_t s_free;                      // group A has read s and t
    uint64_t p_ready, scaled;             // P and dP written; first terms of dq and dk scaled
    uint64_t dv1_full, dv_full, dq_full, out_full;  // k dS; dv; dq; dk, and with it every product
    uint64_t dv_read, dq_read, dk_read;   // their accumulators have been read
    uint64_t dg_done;                     // the sums that dg is made of have been read
    uint64_t tail;                        // rows behind the sequence's end zeroed (blocks that have some)
    uint64_t done;
    float sum;                            // log-decay of the block, times log2(e)
    uint32_t tmem_base;
    int abort_flag;
};

// w[x] of every lane, summed over the warp's lanes: lane l gets the sum of w[l % 16].
__device__ __forceinline__ float warp_column_sums(float (&w)[16]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) {
        const bool up = (lane & off) != 0;
#pragma unroll
        for (int x = 0; x < off; ++x) {
            const float send = up ? w[x] : w[x + off], keep = up ? w[x + off] : w[x];
            w[x] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
    }
    return w[0] + __shfl_xor_sync(0xffffffffu, w[0], 16);
}

template <int D>
__global__ void __launch_bounds__(GatedBackwardCfg<D>::THREADS, 1)
    gated_backward_tc_kernel(const __grid_constant__ GatedBackwardParams p) {
    using C = GatedBackwardCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    GatedBackwardMisc *m = reinterpret_cast<GatedBackwardMisc *>(smem + C::OFF_MISC);
    float *sG = reinterpret_cast<float *>(smem + C::OFF_F);  // gate sums (store_gate_sums)
    float *sR = sG + 128;      // q_i . (first term of dq_i)
    float *sE = sR + 128;      // k_j . (first term of dk_j)
    float *sRow = sE + 128;    // [2][128]: parts of sum_{j < i} W_ij
    float *sCol = sRow + 256;  // [4][128]: parts of sum_{i > j} W_ij, by 32 rows
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    const uint64_t tlimit = p.timeout_ns;
    volatile int *abort_flag = &m->abort_flag;
    const int tiles = p.tab.blocks * p.H;

    if (tid == 0) {
        mbar_init(&m->full_vo, 1);
        mbar_init(&m->full_k, 1);
        mbar_init(&m->full_qs, 1);
        mbar_init(&m->full_ds, 1);
        mbar_init(&m->low_full, 1);
        mbar_init(&m->low_free, 1);
        mbar_init(&m->low_done, 1);
        mbar_init(&m->dv1_full, 1);
        mbar_init(&m->gates, 32);
        mbar_init(&m->first_full, 1);
        mbar_init(&m->dv_full, 1);
        mbar_init(&m->dq_full, 1);
        mbar_init(&m->s_free, C::GROUP_A);
        mbar_init(&m->p_ready, C::GROUP_A);
        mbar_init(&m->scaled, C::GROUP_B);
        mbar_init(&m->out_full, 1);
        mbar_init(&m->dv_read, C::GROUP_A);
        mbar_init(&m->dk_read, C::GROUP_A);
        mbar_init(&m->dq_read, C::GROUP_B);
        mbar_init(&m->dg_done, 32);
        mbar_init(&m->tail, 32);
        mbar_init(&m->done, 1);
        m->abort_flag = 0;
        fence_mbarrier_init_cluster();
        tma_prefetch_desc(&p.tmap_q);
        tma_prefetch_desc(&p.tmap_k);
        tma_prefetch_desc(&p.tmap_v);
        tma_prefetch_desc(&p.tmap_do);
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
    // Loads by warp 0, each as soon as its place is free: dS once k dS is done, v and do once dv
    // is, k once dq is, q and S once dk is; columns of the second parts one after the other.
    int n_ds = 0, n_vo = 0, n_k = 0, n_qs = 0, n_low = 0;
    const int ds_lows = C::STREAM && p.have_ds ? 2 : 0, lows = ds_lows + (C::STREAM && p.have_s ? 2 : 0);
    auto boxes = [&](int to, const CUtensorMap *map, int col, int row, int box, uint64_t *bar) {
#pragma unroll 1
        for (int d = 0; d < C::DB; ++d) tma_load_2d(sbase + to + d * box, map, col + 64 * d, row, bar);
    };
    auto place = [&](int x, int &row, int &col) {
        int rank, blk, start, len, sid;
        p.tab.block(x / p.H, rank, blk);
        p.tab.seqs.get(rank, start, len, sid);
        row = start + blk * C::C;
        col = (x % p.H) * D;
    };
    // part y of tile x's state in a tensor of snapshots
    auto part_row = [](int x, int y) { return (2 * x + y) * D; };
    auto load_ds = [&](int x) {
        ++n_ds;
        if (lane != 0) return;
        mbar_arrive_expect_tx(&m->full_ds, p.have_ds * (C::STREAM ? C::DB : 2) * C::SBOX);
        if (!p.have_ds) return;
        boxes(C::OFF_DS, &p.tmap_ds, 0, part_row(x, 0), C::SBOX, &m->full_ds);
        if (!C::STREAM) boxes(C::OFF_DS + C::SBOX, &p.tmap_ds, 0, part_row(x, 1), C::SBOX, &m->full_ds);
    };
    auto load_low = [&](int x, int i) {
        ++n_low;
        if (lane != 0) return;
        mbar_arrive_expect_tx(&m->low_full, C::SBOX);
        tma_load_2d(sbase + C::OFF_LOW, i < ds_lows ? &p.tmap_ds : &p.tmap_s, 64 * (i & 1), part_row(x, 1),
                    &m->low_full);
    };
    auto load_vo = [&](int row, int col) {
        ++n_vo;
        if (lane != 0) return;
        mbar_arrive_expect_tx(&m->full_vo, 2 * C::TILE);
        boxes(C::OFF_DO, &p.tmap_do, col, row, C::BOX, &m->full_vo);
        boxes(C::OFF_V, &p.tmap_v, col, row, C::BOX, &m->full_vo);
    };
    auto load_k = [&](int row, int col) {
        ++n_k;
        if (lane != 0) return;
        mbar_arrive_expect_tx(&m->full_k, C::TILE);
        boxes(C::OFF_K, &p.tmap_k, col, row, C::BOX, &m->full_k);
    };
    auto load_qs = [&](int x, int row, int col) {
        ++n_qs;
        if (lane != 0) return;
        mbar_arrive_expect_tx(&m->full_qs, C::TILE + p.have_s * (C::STREAM ? C::DB : 2) * C::SBOX);
        boxes(C::OFF_Q, &p.tmap_q, col, row, C::BOX, &m->full_qs);
        if (!p.have_s) return;
        boxes(C::OFF_S, &p.tmap_s, 0, part_row(x, 0), C::SBOX, &m->full_qs);
        if (!C::STREAM) boxes(C::OFF_S + C::SBOX, &p.tmap_s, 0, part_row(x, 1), C::SBOX, &m->full_qs);
    };
    uint32_t raw[4];  // gates of the next tile, fetched ahead (warp 0)
    auto fetch = [&](int x) {
        int rank, blk, start, len, sid;
        p.tab.block(x / p.H, rank, blk);
        p.tab.seqs.get(rank, start, len, sid);
        fetch_gates4(raw, p.g, start + blk * C::C, min(C::C, len - blk * C::C), p.H, x % p.H);
    };
    if (warp == 0 && (int)blockIdx.x < tiles) {
        int row, col;
        place(blockIdx.x, row, col);
        load_vo(row, col);
        load_k(row, col);
        load_qs(blockIdx.x, row, col);
        load_ds(blockIdx.x);
        if (lows > 0) load_low(blockIdx.x, 0);
        fetch(blockIdx.x);
    }
    const uint32_t leader = elect_leader();
    bool ok = true;
    // Phase of the block's barriers, of the block before, and of `tail`.  Every wait is exact: no
    // barrier's next phase completes before all who wait for this one have returned.  Each load
    // of the next block needs a product of this one behind p_ready, hence group A's waits (and
    // the last one scaled, hence group B's); the next block's products need dv_read, dq_read and
    // dk_read; its sums (p_ready, scaled) dg_done.
    uint32_t ph = 0, tail_ph = 0, low_ph = 0;
    for (int x = blockIdx.x; ok && x < tiles; x += gridDim.x, ph ^= 1u) {
        const int h = x % p.H;
        int rank, blk, start, len, sid;
        p.tab.block(x / p.H, rank, blk);
        p.tab.seqs.get(rank, start, len, sid);
        const int row0 = start + blk * C::C, nv = min(C::C, len - blk * C::C);
        const int next = x + (int)gridDim.x;
        const bool first = x == (int)blockIdx.x, tail = nv < C::C;
        if (warp == 0) {
            // ------------------------------------------------------------ gate sums, loads
            float gate[4];
            widen_gates4(gate, raw);
            store_gate_sums(sG, &m->sum, gate);
            mbar_arrive(&m->gates);
            if (tail) {
                // rows of the next sequence must not enter any sum over the block's tokens
                ok = wwait(&m->full_qs, ph) && wwait(&m->full_k, ph) && wwait(&m->full_vo, ph);
                if (!ok) break;
                for (int t = 0; t < 4 * C::DB; ++t)
                    for (int c = nv * 8 + lane; c < C::C * 8; c += 32)
                        st_shared_v4(sbase + t * C::BOX + c * 16, 0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
                mbar_arrive(&m->tail);
            }
            // low_free of a load needs low_full, its wait and its product; the next phase this load
            for (int i = 1; ok && i <= lows; ++i, low_ph ^= 1u) {
                if (i == lows && next >= tiles) break;
                if ((ok = wwait(&m->low_free, low_ph))) load_low(i < lows ? x : next, i < lows ? i : 0);
            }
            if (ok && next < tiles) {
                int row, col;
                place(next, row, col);
                fetch(next);
                if ((ok = wwait(&m->dv1_full, ph))) load_ds(next);
                if (ok && (ok = wwait(&m->dv_full, ph))) load_vo(row, col);
                if (ok && (ok = wwait(&m->dq_full, ph))) load_k(row, col);
                if (ok && (ok = wwait(&m->out_full, ph))) load_qs(next, row, col);
            }
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issue
            // a row-major tile is read along its columns (kk: 64-column boxes of 128 rows, ss:
            // of D rows) or, transposed, along its rows (nn)
            auto kk = [](int ks) { return (uint32_t)((ks >> 2) * C::BOX + (ks & 3) * 32); };
            auto ss = [](int ks) { return (uint32_t)((ks >> 2) * C::SBOX + (ks & 3) * 32); };
            auto nn = [](int ks) { return (uint32_t)(ks * 2048); };
            // D (+)= A B over n steps of 16; `keep` adds to what D holds
            auto product = [&](uint32_t d, uint64_t a, auto at_a, uint64_t b, auto at_b, uint32_t id, int n,
                               bool keep) {
#pragma unroll 2
                for (int ks = 0; ks < n; ++ks)
                    warp_mma_ss(leader, tmem + d, desc_add(a, at_a(ks)), desc_add(b, at_b(ks)), id,
                                keep || ks > 0 ? 1u : 0u);
            };
            const uint64_t qk = desc_kmajor_sw128(sbase + C::OFF_Q), kkd = desc_kmajor_sw128(sbase + C::OFF_K),
                           vk = desc_kmajor_sw128(sbase + C::OFF_V), ok_ = desc_kmajor_sw128(sbase + C::OFF_DO);
            ok = wwait(&m->full_vo, ph) && (!tail || wwait(&m->tail, tail_ph)) && (first || wwait(&m->dv_read, ph ^ 1u));
            if (ok) {
                tc_fence_after();
                product(C::TM_T, ok_, kk, vk, kk, C::ID_S, D / 16, false);
                ok = wwait(&m->full_ds, ph) && (first || wwait(&m->dk_read, ph ^ 1u));
            }
            // STREAM: d += a B^T, 64 columns `half` of a and of the second part of B
            auto low = [&](uint32_t d, uint64_t a, int half, bool keep) {
                if (!(ok = ok && wwait(&m->low_full, low_ph))) return;
                tc_fence_after();
                product(d, desc_add(a, half * C::BOX), kk, desc_kmajor_sw128(sbase + C::OFF_LOW), ss, C::ID_KK, 4, keep);
                warp_commit(leader, &m->low_free);
                low_ph ^= 1u;
            };
            if (ok) {
                tc_fence_after();
                if (p.have_ds) {
                    product(C::TM_DK, vk, kk, desc_kmajor_sw128(sbase + C::OFF_DS), ss, C::ID_KK, D / 16, false);
                    if (!C::STREAM)
                        product(C::TM_DK, vk, kk, desc_kmajor_sw128(sbase + C::OFF_DS + C::SBOX), ss, C::ID_KK, D / 16,
                                true);
                    else
                        low(C::TM_DK, vk, 0, true);
                }
                ok = ok && wwait(&m->full_k, ph) && wwait(&m->full_qs, ph);
            }
            if (ok) {
                tc_fence_after();
                product(C::TM_S, qk, kk, kkd, kk, C::ID_S, D / 16, false);
                ok = first || wwait(&m->dq_read, ph ^ 1u);
            }
            if (ok) {
                tc_fence_after();
                if (p.have_s) {
                    product(C::TM_DQ, ok_, kk, desc_kmajor_sw128(sbase + C::OFF_S), ss, C::ID_KK, D / 16, false);
                    if (!C::STREAM)
                        product(C::TM_DQ, ok_, kk, desc_kmajor_sw128(sbase + C::OFF_S + C::SBOX), ss, C::ID_KK, D / 16,
                                true);
                }
                if (ds_lows > 0) low(C::TM_DK, vk, 1, true);
            }
            if (ok) {
                warp_commit(leader, &m->first_full);
                if (C::STREAM && p.have_s) {
                    low(C::TM_DQ, ok_, 0, true);
                    low(C::TM_DQ, ok_, 1, true);
                    if (ok) warp_commit(leader, &m->low_done);
                }
            }
            if (ok) {
                ok = wwait(&m->s_free, ph);
            }
            if (ok) {
                tc_fence_after();
                if (p.have_ds)
                    product(C::TM_DV1, kkd, kk, desc_mnmajor_sw128(sbase + C::OFF_DS, C::SBOX), nn, C::ID_KN, D / 16,
                            false);
                warp_commit(leader, &m->dv1_full);
                ok = wwait(&m->p_ready, ph);
            }
            if (ok) {
                tc_fence_after();
                product(C::TM_DV2, desc_mnmajor_sw128(sbase + C::OFF_P, C::BOX), nn,
                        desc_mnmajor_sw128(sbase + C::OFF_DO, C::BOX), nn, C::ID_NN, C::C / 16, false);
                warp_commit(leader, &m->dv_full);
                ok = wwait(&m->scaled, ph);
            }
            if (ok) {
                tc_fence_after();
                product(C::TM_DQ, desc_kmajor_sw128(sbase + C::OFF_DP), kk, desc_mnmajor_sw128(sbase + C::OFF_K, C::BOX),
                        nn, C::ID_KN, C::C / 16, p.have_s != 0);
                warp_commit(leader, &m->dq_full);
                product(C::TM_DK, desc_mnmajor_sw128(sbase + C::OFF_DP, C::BOX), nn,
                        desc_mnmajor_sw128(sbase + C::OFF_Q, C::BOX), nn, C::ID_NN, C::C / 16, p.have_ds != 0);
                warp_commit(leader, &m->out_full);
            }
            __syncwarp();
        } else if (warp == 14) {
            // ------------------------------------------------------------ dg
            float part = 0.f;
            if (p.through != nullptr && lane < 8 * C::DB) part = p.through[(size_t)x * (8 * C::DB) + lane];
            ok = wwait(&m->p_ready, ph) && wwait(&m->scaled, ph);
            if (!ok) break;
            float r[4], e[4], up[4], down[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int t = 4 * lane + y;
                r[y] = sR[t];
                e[y] = sE[t] + (((sCol[t] + sCol[128 + t]) + (sCol[256 + t] + sCol[384 + t])) -
                                (sRow[t] + sRow[128 + t]));
            }
            reads_done();
            mbar_arrive(&m->dg_done);
            if (p.dg != nullptr) {
                // dg_t = e^{G_C} <dS, S> + sum_{i >= t} sR_i + sum_{j < t} (sE_j + col_j - row_j)
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) part += __shfl_xor_sync(0xffffffffu, part, off);
                prefix_gates4(e, down);   // down[y] = sum_{j <= t}
                suffix_gates4(r, up);     // up[y] = sum_{i > t}
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int t = 4 * lane + y;
                    if (t < nv)
                        p.dg[(size_t)(row0 + t) * p.H + h] =
                            __float2bfloat16_rn(part + (up[y] + r[y]) + (down[y] - e[y]));
                }
            }
            __syncwarp();
        } else {
            const int q = warp & 3;
            const int i = 32 * q + lane;                       // this thread's row
            const uint32_t lanes = (uint32_t)(32 * q) << 16;
            const bool A = warp < 2 + C::GROUP_A / 32;
            const int half = A ? (warp - 2) >> 2 : 0;
            // 64 columns of this warp's rows out of TMEM and into `out`; with `twice`, dv's first
            // term times w is added.  32 columns at a time pass through the warp's 1 KB of shared
            // memory, 16 rows at a time (rows of 64 bytes, chunk c of row r at c ^ (r / 2 % 4)), to be
            // stored eight rows at a time: from registers a store would touch 32 rows, 32 passes of the
            // memory pipe.
            const uint32_t stage = sbase + C::OFF_STAGE + (warp - 2) * 1024;
            auto store = [&](uint32_t col, bool twice, float w, __nv_bfloat16 *out, int box) {
#pragma unroll 1
                for (int cc = 0; cc < 2; ++cc) {
                    uint32_t a[32];
                    tmem_ld32(tmem + col + 64 * box + 32 * cc + lanes, a);
                    if (twice) {
                        uint32_t b[32];
                        tmem_ld32(tmem + C::TM_DV1 + 64 * box + 32 * cc + lanes, b);
                        tmem_ld_wait();
#pragma unroll
                        for (int y = 0; y < 32; ++y)
                            a[y] = __float_as_uint(fmaf(w, __uint_as_float(b[y]), __uint_as_float(a[y])));
                    }
                    tmem_ld_wait();
                    const int r0 = lane >> 2, c = lane & 3;
                    __nv_bfloat16 *dst =
                        out + ((size_t)(row0 + 32 * q + r0) * p.H + h) * D + 64 * box + 32 * cc + 8 * c;
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        __syncwarp();  // the last pass has been read back
                        if (lane >> 4 == z) {
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                st_shared_v4(stage + (lane & 15) * 64 + ((y ^ ((lane >> 1) & 3)) << 4),
                                             pack_bf16x2(__uint_as_float(a[8 * y]), __uint_as_float(a[8 * y + 1])),
                                             pack_bf16x2(__uint_as_float(a[8 * y + 2]), __uint_as_float(a[8 * y + 3])),
                                             pack_bf16x2(__uint_as_float(a[8 * y + 4]), __uint_as_float(a[8 * y + 5])),
                                             pack_bf16x2(__uint_as_float(a[8 * y + 6]), __uint_as_float(a[8 * y + 7])));
                        }
                        __syncwarp();
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int r = 8 * y + r0;  // of the 16
                            const uint4 v = ld_shared_v4(stage + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
                            if (32 * q + 16 * z + r < nv)
                                *reinterpret_cast<uint4 *>(dst + (size_t)(16 * z + 8 * y) * p.H * D) = v;
                        }
                    }
                }
            };
            if (A) {
                // -------------------------------------------------------- group A: P, dP, W
                // (behind first_full v and S have been read: P and dP may take their places)
                ok = wwait(&m->gates, ph) && wwait(&m->first_full, ph) && (first || wwait(&m->dg_done, ph ^ 1u));
                float wt = 0.f;
                if (ok) {
                    tc_fence_after();
                    const uint32_t si = __float_as_uint(sG[i]);
                    const uint64_t s2 = pair_f32(si, si);
                    wt = ex2(sG[i]);
                    float row = 0.f;
#pragma unroll 1
                    for (int pc = half; pc < 8; pc += 2) {     // every other 16 columns
                        uint32_t P[8], dP[8];                  // packed
                        float col = 0.f;
                        if (pc <= 2 * q + 1) {                 // columns that rows of this warp see
                            uint32_t sc[16], t[16];
                            tmem_ld16(tmem + C::TM_S + 16 * pc + lanes, sc);
                            tmem_ld16(tmem + C::TM_T + 16 * pc + lanes, t);
                            tmem_ld_wait();
                            if (pc >= 2 * q) {  // the warp's last columns of s and t
                                tc_fence_before();
                                mbar_arrive(&m->s_free);
                            }
                            uint64_t w2[8], sum2 = 0;          // W in pairs of columns
#pragma unroll
                            for (int y = 0; y < 16; y += 4) {
                                const ulonglong2 sj = *reinterpret_cast<const ulonglong2 *>(&sG[16 * pc + y]);
#pragma unroll
                                for (int z = 0; z < 4; z += 2) {
                                    const uint64_t d = ex2_f32x2(sub_f32x2(z == 0 ? sj.x : sj.y, s2));
                                    const uint64_t tt = pair_f32(t[y + z], t[y + z + 1]);
                                    const uint64_t pp = mul_f32x2(pair_f32(sc[y + z], sc[y + z + 1]), d);
                                    P[(y + z) / 2] = pack_f32x2(pp);
                                    dP[(y + z) / 2] = pack_f32x2(mul_f32x2(tt, d));
                                    w2[(y + z) / 2] = mul_f32x2(pp, tt);
                                }
                            }
                            if (pc >= 2 * q) {  // columns behind this row, whatever they hold, give 0
                                const int seen = i - 16 * pc;  // columns before this row
#pragma unroll
                                for (int y = 0; y < 8; ++y) {
                                    const uint32_t m0 = 2 * y <= seen ? 0xffffffffu : 0u,
                                                   m1 = 2 * y + 1 <= seen ? 0xffffffffu : 0u,
                                                   m2 = 2 * y + 2 <= seen ? 0xffffffffu : 0u;
                                    P[y] &= (m0 & 0xffffu) | (m1 & 0xffff0000u);
                                    dP[y] &= (m0 & 0xffffu) | (m1 & 0xffff0000u);
                                    w2[y] &= (uint64_t)m1 | ((uint64_t)m2 << 32);  // j < i
                                }
                            }
                            float w[16];
#pragma unroll
                            for (int y = 0; y < 8; ++y) {
                                sum2 = add_f32x2(sum2, w2[y]);
                                w[2 * y] = __uint_as_float((uint32_t)w2[y]);
                                w[2 * y + 1] = __uint_as_float((uint32_t)(w2[y] >> 32));
                            }
                            row += __uint_as_float((uint32_t)sum2) + __uint_as_float((uint32_t)(sum2 >> 32));
                            col = warp_column_sums(w);
                        } else {
#pragma unroll
                            for (int y = 0; y < 8; ++y) P[y] = dP[y] = 0u;
                        }
                        if (lane < 16) sCol[128 * q + 16 * pc + lane] = col;
                        const uint32_t at = sbase + (uint32_t)((pc >> 2) * C::BOX + i * 128);
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const uint32_t o = at + (((2 * (pc & 3) + c) ^ (i & 7)) << 4);
                            st_shared_v4(C::OFF_P + o, P[4 * c], P[4 * c + 1], P[4 * c + 2], P[4 * c + 3]);
                            st_shared_v4(C::OFF_DP + o, dP[4 * c], dP[4 * c + 1], dP[4 * c + 2], dP[4 * c + 3]);
                        }
                    }
                    sRow[128 * half + i] = row;
                    fence_proxy_async_smem();
                    mbar_arrive(&m->p_ready);
                    ok = wwait(&m->dv_full, ph);
                }
                // results: dv while the products of dq and dk run, then dk
#pragma unroll 1
                for (int n = 0; ok && n < 2; ++n) {
                    if (n == 1) ok = wwait(&m->out_full, ph);
                    if (!ok) break;
                    tc_fence_after();
                    if (half < C::DB)
                        store(n == 0 ? C::TM_DV2 : C::TM_DK, n == 0 && p.have_ds != 0, wt, n == 0 ? p.dv : p.dk, half);
                    tc_fence_before();
                    mbar_arrive(n == 0 ? &m->dv_read : &m->dk_read);
                }
            } else {
                // -------------------------------------------------------- group B: first terms
                float r = 0.f, e = 0.f;
                ok = wwait(&m->gates, ph) && wwait(&m->full_qs, ph) && wwait(&m->full_k, ph) &&
                     wwait(&m->first_full, ph) &&
                     (!tail || wwait(&m->tail, tail_ph)) && (first || wwait(&m->dg_done, ph ^ 1u));
                if (ok) {
                    tc_fence_after();
                    // rows of accumulators times w; their product with a row of q or k
                    auto scale = [&](uint32_t col, float w, int tile, float &dot) {
#pragma unroll 1
                        for (int cc = 0; cc < D / 32; ++cc) {
                            uint32_t a[32];
                            tmem_ld32(tmem + col + 32 * cc + lanes, a);
                            tmem_ld_wait();
#pragma unroll
                            for (int y = 0; y < 32; ++y) a[y] = __float_as_uint(w * __uint_as_float(a[y]));
                            tmem_st32(tmem + col + 32 * cc + lanes, a);
                            float d0 = 0.f, d1 = 0.f;
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const int ch = (cc & 1) * 4 + c;
                                const uint4 v = ld_shared_v4(sbase + tile + (cc >> 1) * C::BOX + i * 128 +
                                                             ((ch ^ (i & 7)) << 4));
                                const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int z = 0; z < 4; ++z) {
                                    d0 = fmaf(__uint_as_float(in[z] << 16), __uint_as_float(a[8 * c + 2 * z]), d0);
                                    d1 = fmaf(__uint_as_float(in[z] & 0xffff0000u),
                                              __uint_as_float(a[8 * c + 2 * z + 1]), d1);
                                }
                            }
                            dot += d0 + d1;
                        }
                    };
                    // e^{G_i}, e^{G_C - G_i}
                    const float up = ex2(m->sum - sG[i]), down = ex2(sG[i]);
                    if (p.have_ds) scale(C::TM_DK, down, C::OFF_K, e);
                    if (C::STREAM && p.have_s) {
                        ok = wwait(&m->low_done, ph);
                        tc_fence_after();
                    }
                    if (p.have_s) scale(C::TM_DQ, up, C::OFF_Q, r);
                    sR[i] = r;
                    sE[i] = e;
                    tmem_st_wait();
                    tc_fence_before();
                    // the products that wait for this arrival let TMA take the places of q and k,
                    // whose rows were read above
                    fence_proxy_async_smem();
                    mbar_arrive(&m->scaled);
                    ok = ok && wwait(&m->dq_full, ph);
                }
                if (ok) {
                    tc_fence_after();
#pragma unroll 1
                    for (int n = 0; n < C::DB; ++n) store(C::TM_DQ, false, 0.f, p.dq, n);
                    tc_fence_before();
                    mbar_arrive(&m->dq_read);
                }
            }
        }
        if (tail) tail_ph ^= 1u;
    }
    if (!ok) fail();
    if (warp == 0 && !ok) {  // loads that are still in flight land before the CTA ends
        auto landed = [&](uint64_t *bar, int n) {
            if (n > 0) mbar_wait(bar, (uint32_t)((n - 1) & 1), nullptr, tlimit);
        };
        landed(&m->full_ds, n_ds);
        landed(&m->low_full, n_low);
        landed(&m->full_vo, n_vo);
        landed(&m->full_k, n_k);
        landed(&m->full_qs, n_qs);
    }
    if (warp == 1) {  // every issued MMA has finished before TMEM is freed
        warp_commit(leader, &m->done);
        mbar_wait(&m->done, 0u, nullptr, tlimit);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace la
