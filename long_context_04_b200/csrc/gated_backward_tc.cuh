// Gradients of gated lightning attention on the tensor cores (bf16), one block of 128 tokens
// of one head at a time: from the bf16 state S at the block's start and the gradient dS of
// the state at its end (the state scans' snapshots), every block stands alone.
//
//   scores   s = q k^T, t = do v^T;  P = s (.) decay,  dP = t (.) decay     (j <= i)
//   dq = e^{G_i} (do S^T)        + dP k
//   dk = e^{G_C - G_j} (v dS^T)  + dP^T q
//   dv = e^{G_C - G_j} (k dS)    + P^T do
//   dg as in gated.cuh, from W = dP (.) s and the row sums of q . dq and k . dk of the first
//   terms.
//
// A persistent CTA per SM (192 KB of tiles: q, k, v, do and S, dS, whose place P and dP take
// once the products that read S and dS are done).  TMEM, 512 columns: s, t, dq, dk; dv takes
// the place of s.  The decays of the first terms differ by row, so their products go to TMEM,
// are scaled there, and the second products accumulate on top.  Eight products per block:
//   s, t; do S^T, v dS^T; k dS  ->  scaling, P, dP  ->  dP k, dP^T q, P^T do.
// P and dP are each stored once, [i][j]: as the left factor of dP k they are read along j, as
// the transposed left factor of the other two along i.
//
// Warps: 0 TMA loads, gates and dg; 1 MMA issue; 2-5 (group A) scores -> P, dP, W; 6-9
// (group B) scaling of the first terms and their row sums.  Both groups store the results.
// Every barrier completes one phase per block, and all warps meet at the block's end.
//
// HBM: 14 D bytes of tiles and results and 4 D^2 / 128 bytes of snapshots per token and head.
#pragma once

#include "gated_state_tc.cuh"

namespace la {

struct GatedBackwardParams {
    CUtensorMap tmap_q, tmap_k, tmap_v, tmap_do;  // [T][H*D], box 64 x 128
    CUtensorMap tmap_s, tmap_ds;                  // [blocks * H * D][D], box 64 x D
    const __nv_bfloat16 *g;
    const float *through;  // [blocks][H][4 D / 64] parts of e^{G_C} <dS, S>, or nullptr
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
    static constexpr int OFF_Q = 0, OFF_K = TILE, OFF_V = 2 * TILE, OFF_DO = 3 * TILE;
    static constexpr int OFF_P = 4 * TILE, OFF_DP = OFF_P + PT;   // P over S, dP over dS
    static constexpr int OFF_F = OFF_DP + PT;   // 10 arrays of 128 floats
    static constexpr int OFF_MISC = OFF_F + 10 * 512;
    static constexpr int SMEM_BYTES = 1024 + OFF_MISC + 512;
    static_assert(DB * SBOX <= PT, "a state fits into the place of P");
    static_assert(SMEM_BYTES > 114 * 1024 && SMEM_BYTES <= 227 * 1024, "one CTA per SM");
    static constexpr int TM_S = 0, TM_T = 128, TM_DQ = 256, TM_DK = 384, TM_DV = 0;
    static constexpr int THREADS = 64 + 256;
    static constexpr uint32_t ID_S = idesc_bf16_f32(128, 128, 0, 0);
    static constexpr uint32_t ID_KK = idesc_bf16_f32(128, D, 0, 0);
    static constexpr uint32_t ID_KN = idesc_bf16_f32(128, D, 0, 1);
    static constexpr uint32_t ID_NN = idesc_bf16_f32(128, D, 1, 1);
};

struct GatedBackwardMisc {
    uint64_t full_qk, full_vo, full_ss;   // tiles landed
    uint64_t gates;                       // decays of the block written
    uint64_t s_full, first_full, dv_full; // s and t; do S^T and v dS^T; k dS
    uint64_t s_free;                      // group A has read s
    uint64_t p_ready, scaled, out_full;
    uint64_t done;
    uint32_t tmem_base;
    int abort_flag;
};

// w[x] of every lane, summed over the warp's lanes: lane l gets the sum of w[l].
__device__ __forceinline__ float warp_column_sums(float (&w)[32]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const bool up = (lane & off) != 0;
#pragma unroll
        for (int x = 0; x < off; ++x) {
            const float send = up ? w[x] : w[x + off], keep = up ? w[x + off] : w[x];
            w[x] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
    }
    return w[0];
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
    float *sG2 = reinterpret_cast<float *>(smem + C::OFF_F);  // G_i log2(e)
    float *sGam = sG2 + 128;   // e^{G_i}
    float *sWt = sGam + 128;   // e^{G_C - G_j}
    float *sR = sWt + 128;     // q_i . (first term of dq_i)
    float *sE = sR + 128;      // k_j . (first term of dk_j)
    float *sRow = sE + 128;    // sum_{j < i} W_ij
    float *sCol = sRow + 128;  // [4][128]: each warp's part of sum_{i > j} W_ij
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    const uint64_t tlimit = p.timeout_ns;
    volatile int *abort_flag = &m->abort_flag;
    const int tiles = p.tab.blocks * p.H;

    if (tid == 0) {
        mbar_init(&m->full_qk, 1);
        mbar_init(&m->full_vo, 1);
        mbar_init(&m->full_ss, 1);
        mbar_init(&m->gates, 32);
        mbar_init(&m->s_full, 1);
        mbar_init(&m->first_full, 1);
        mbar_init(&m->dv_full, 1);
        mbar_init(&m->s_free, 128);
        mbar_init(&m->p_ready, 128);
        mbar_init(&m->scaled, 128);
        mbar_init(&m->out_full, 1);
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
    auto fail = [&]() {
        *abort_flag = 1;
        record_fault(DEV_TIMEOUT);
    };
    auto wwait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return warp_wait(bar, parity, abort_flag, tlimit);
    };
    uint32_t load_phase = 1;      // of thread 0: the phase of its last loads
    auto load = [&](int x) {      // thread 0: the tiles of tile x
        load_phase ^= 1u;
        int rank, blk, start, len, sid;
        p.tab.block(x / p.H, rank, blk);
        p.tab.seqs.get(rank, start, len, sid);
        const int row = start + blk * C::C, col = (x % p.H) * D;
        mbar_arrive_expect_tx(&m->full_qk, 2 * C::TILE);
        for (int d = 0; d < C::DB; ++d) {
            tma_load_2d(sbase + C::OFF_Q + d * C::BOX, &p.tmap_q, col + 64 * d, row, &m->full_qk);
            tma_load_2d(sbase + C::OFF_K + d * C::BOX, &p.tmap_k, col + 64 * d, row, &m->full_qk);
        }
        mbar_arrive_expect_tx(&m->full_vo, 2 * C::TILE);
        for (int d = 0; d < C::DB; ++d) {
            tma_load_2d(sbase + C::OFF_DO + d * C::BOX, &p.tmap_do, col + 64 * d, row, &m->full_vo);
            tma_load_2d(sbase + C::OFF_V + d * C::BOX, &p.tmap_v, col + 64 * d, row, &m->full_vo);
        }
        mbar_arrive_expect_tx(&m->full_ss, (p.have_s + p.have_ds) * C::DB * C::SBOX);
        for (int d = 0; d < C::DB; ++d) {
            if (p.have_s) tma_load_2d(sbase + C::OFF_P + d * C::SBOX, &p.tmap_s, 64 * d, x * D, &m->full_ss);
            if (p.have_ds) tma_load_2d(sbase + C::OFF_DP + d * C::SBOX, &p.tmap_ds, 64 * d, x * D, &m->full_ss);
        }
    };

    if (tid == 0 && (int)blockIdx.x < tiles) load(blockIdx.x);
    bool ok = true;
    uint32_t ph = 0;
    for (int x = blockIdx.x; x < tiles; x += gridDim.x, ph ^= 1u) {
        const int h = x % p.H;
        int rank, blk, start, len, sid;
        p.tab.block(x / p.H, rank, blk);
        p.tab.seqs.get(rank, start, len, sid);
        const int row0 = start + blk * C::C, nv = min(C::C, len - blk * C::C);
        if (nv < C::C) {
            // rows of the next sequence must not enter any sum over the block's tokens
            if (ok) ok = wwait(&m->full_qk, ph) && wwait(&m->full_vo, ph);
            for (int t = 0; t < 4 * C::DB; ++t)
                for (int c = nv * 8 + tid; c < C::C * 8; c += C::THREADS)
                    st_shared_v4(sbase + t * C::BOX + c * 16, 0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncthreads();
        }
        if (warp == 0) {
            // ------------------------------------------------------------ gates, loads, dg
            uint32_t raw[4];
            float gate[4], sums[4], aft[4];
            fetch_gates4(raw, p.g, row0, nv, p.H, h);
            widen_gates4(gate, raw);
            prefix_gates4(gate, sums);
            suffix_gates4(gate, aft);
            float part = 0.f;
            if (p.through != nullptr && lane < 4 * C::DB) part = p.through[(size_t)x * (4 * C::DB) + lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sG2[4 * lane + e] = sums[e] * 1.4426950408889634f;
                sGam[4 * lane + e] = expf(sums[e]);
                sWt[4 * lane + e] = expf(aft[e]);
            }
            mbar_arrive(&m->gates);
            if (ok) ok = wwait(&m->out_full, ph);
            // every product that reads the tiles is done
            if (ok && lane == 0 && x + (int)gridDim.x < tiles) load(x + gridDim.x);
            // group A's and group B's sums were written before the products of out_full were
            // issued, but this warp has to see them itself
            if (ok) ok = wwait(&m->p_ready, ph) && wwait(&m->scaled, ph);
            if (ok && p.dg != nullptr) {
                // dg_t = e^{G_C} <dS, S> + sum_{i >= t} sR_i + sum_{j < t} (sE_j + col_j - row_j)
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) part += __shfl_xor_sync(0xffffffffu, part, off);
                float r[4], e[4], up[4], down[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int t = 4 * lane + y;
                    r[y] = sR[t];
                    e[y] = sE[t] + (((sCol[t] + sCol[128 + t]) + (sCol[256 + t] + sCol[384 + t])) - sRow[t]);
                }
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
                mma_bf16_ss(tmem + d, desc_add(a, at_a(0)), desc_add(b, at_b(0)), id, keep ? 1u : 0u);
#pragma unroll
                for (int ks = 1; ks < n; ++ks)
                    mma_bf16_ss(tmem + d, desc_add(a, at_a(ks)), desc_add(b, at_b(ks)), id, 1u);
            };
            const uint64_t qk = desc_kmajor_sw128(sbase + C::OFF_Q), kkd = desc_kmajor_sw128(sbase + C::OFF_K),
                           vk = desc_kmajor_sw128(sbase + C::OFF_V), ok_ = desc_kmajor_sw128(sbase + C::OFF_DO);
            if (ok) ok = wwait(&m->full_qk, ph);
            if (ok) {
                tc_fence_after();
                if (lane == 0) product(C::TM_S, qk, kk, kkd, kk, C::ID_S, D / 16, false);
                __syncwarp();
                ok = wwait(&m->full_vo, ph);
            }
            if (ok) {
                tc_fence_after();
                if (lane == 0) {
                    product(C::TM_T, ok_, kk, vk, kk, C::ID_S, D / 16, false);
                    mma_commit(&m->s_full);
                }
                __syncwarp();
                ok = wwait(&m->full_ss, ph);
            }
            if (ok) {
                tc_fence_after();
                // (Uniform branches around the elected thread's, not inside it: nested the other
                // way, the first product instruction behind the inner test went missing at D = 64.)
                if (p.have_s) {
                    if (lane == 0)
                        product(C::TM_DQ, ok_, kk, desc_kmajor_sw128(sbase + C::OFF_P), ss, C::ID_KK, D / 16, false);
                    __syncwarp();
                }
                if (p.have_ds) {
                    if (lane == 0)
                        product(C::TM_DK, vk, kk, desc_kmajor_sw128(sbase + C::OFF_DP), ss, C::ID_KK, D / 16, false);
                    __syncwarp();
                }
                if (lane == 0) mma_commit(&m->first_full);
                __syncwarp();
                ok = wwait(&m->s_free, ph);
            }
            if (ok) {
                tc_fence_after();
                if (p.have_ds) {
                    if (lane == 0)
                        product(C::TM_DV, kkd, kk, desc_mnmajor_sw128(sbase + C::OFF_DP, C::SBOX), nn, C::ID_KN,
                                D / 16, false);
                    __syncwarp();
                }
                if (lane == 0) mma_commit(&m->dv_full);
                __syncwarp();
                ok = wwait(&m->p_ready, ph) && wwait(&m->scaled, ph);
            }
            if (ok) {
                tc_fence_after();
                if (lane == 0) {
                    const uint64_t dpk = desc_kmajor_sw128(sbase + C::OFF_DP),
                                   dpn = desc_mnmajor_sw128(sbase + C::OFF_DP, C::BOX),
                                   pn = desc_mnmajor_sw128(sbase + C::OFF_P, C::BOX),
                                   qn = desc_mnmajor_sw128(sbase + C::OFF_Q, C::BOX),
                                   kn = desc_mnmajor_sw128(sbase + C::OFF_K, C::BOX),
                                   on = desc_mnmajor_sw128(sbase + C::OFF_DO, C::BOX);
                    product(C::TM_DQ, dpk, kk, kn, nn, C::ID_KN, C::C / 16, p.have_s != 0);
                    product(C::TM_DK, dpn, nn, qn, nn, C::ID_NN, C::C / 16, p.have_ds != 0);
                    product(C::TM_DV, pn, nn, on, nn, C::ID_NN, C::C / 16, p.have_ds != 0);
                    mma_commit(&m->out_full);
                }
                __syncwarp();
            }
        } else {
            const int q = warp & 3;
            const int i = 32 * q + lane;                       // this thread's row
            const uint32_t lanes = (uint32_t)(32 * q) << 16;
            if (warp < 6) {
                // -------------------------------------------------------- group A: P, dP, W
                uint32_t pp[64], dd[64];                       // packed rows of P and dP
                if (ok) ok = wwait(&m->gates, ph) && wwait(&m->s_full, ph);
                if (ok) {
                    tc_fence_after();
                    const float Gi = sG2[i];
                    float row = 0.f;
#pragma unroll
                    for (int cc = 0; cc < 4; ++cc) {
                        if (cc <= q) {                         // columns that the rows of this warp see
                            uint32_t s[32], t[32];
                            tmem_ld32(tmem + C::TM_S + 32 * cc + lanes, s);
                            tmem_ld32(tmem + C::TM_T + 32 * cc + lanes, t);
                            tmem_ld_wait();
                            float w[32];
#pragma unroll
                            for (int y = 0; y < 32; y += 4) {
                                const float4 Gj = *reinterpret_cast<const float4 *>(&sG2[32 * cc + y]);
                                const float gj[4] = {Gj.x, Gj.y, Gj.z, Gj.w};
                                float P[4], dP[4];
#pragma unroll
                                for (int z = 0; z < 4; ++z) {
                                    const bool seen = cc < q || y + z <= lane;
                                    const float d = ex2(Gi - gj[z]);
                                    P[z] = seen ? __uint_as_float(s[y + z]) * d : 0.f;
                                    dP[z] = seen ? __uint_as_float(t[y + z]) * d : 0.f;
                                    w[y + z] = cc < q || y + z < lane ? P[z] * __uint_as_float(t[y + z]) : 0.f;
                                    row += w[y + z];
                                }
                                pp[16 * cc + y / 2] = pack_bf16x2(P[0], P[1]);
                                pp[16 * cc + y / 2 + 1] = pack_bf16x2(P[2], P[3]);
                                dd[16 * cc + y / 2] = pack_bf16x2(dP[0], dP[1]);
                                dd[16 * cc + y / 2 + 1] = pack_bf16x2(dP[2], dP[3]);
                            }
                            sCol[128 * q + 32 * cc + lane] = warp_column_sums(w);
                        } else {
#pragma unroll
                            for (int y = 0; y < 16; ++y) pp[16 * cc + y] = dd[16 * cc + y] = 0u;
                            sCol[128 * q + 32 * cc + lane] = 0.f;
                        }
                    }
                    sRow[i] = row;
                    tc_fence_before();
                    mbar_arrive(&m->s_free);
                    // the products that read S and dS are done: their place is free
                    ok = wwait(&m->first_full, ph) && wwait(&m->dv_full, ph);
                }
                if (ok) {
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const uint32_t at = (uint32_t)((c >> 3) * C::BOX + i * 128 + (((c & 7) ^ (i & 7)) << 4));
                        st_shared_v4(sbase + C::OFF_P + at, pp[4 * c], pp[4 * c + 1], pp[4 * c + 2], pp[4 * c + 3]);
                        st_shared_v4(sbase + C::OFF_DP + at, dd[4 * c], dd[4 * c + 1], dd[4 * c + 2], dd[4 * c + 3]);
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(&m->p_ready);
                }
            } else {
                // -------------------------------------------------------- group B: first terms
                float r = 0.f, e = 0.f;
                if (ok) ok = wwait(&m->gates, ph) && wwait(&m->full_qk, ph) && wwait(&m->first_full, ph);
                if (ok) {
                    tc_fence_after();
                    // rows of D accumulators times w; their product with a row of q or k
                    auto scale = [&](uint32_t col, float w, int tile, float &dot) {
#pragma unroll 1
                        for (int cc = 0; cc < D / 32; ++cc) {
                            uint32_t a[32];
                            tmem_ld32(tmem + col + 32 * cc + lanes, a);
                            tmem_ld_wait();
#pragma unroll
                            for (int y = 0; y < 32; ++y) a[y] = __float_as_uint(w * __uint_as_float(a[y]));
                            tmem_st32(tmem + col + 32 * cc + lanes, a);
                            if (tile >= 0) {
#pragma unroll
                                for (int c = 0; c < 4; ++c) {
                                    const int ch = (cc & 1) * 4 + c;
                                    const uint4 v = ld_shared_v4(sbase + tile + (cc >> 1) * C::BOX + i * 128 +
                                                                 ((ch ^ (i & 7)) << 4));
                                    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                    for (int z = 0; z < 4; ++z) {
                                        dot = fmaf(__uint_as_float(in[z] << 16), __uint_as_float(a[8 * c + 2 * z]), dot);
                                        dot = fmaf(__uint_as_float(in[z] & 0xffff0000u),
                                                   __uint_as_float(a[8 * c + 2 * z + 1]), dot);
                                    }
                                }
                            }
                        }
                    };
                    float none = 0.f;
                    if (p.have_s) scale(C::TM_DQ, sGam[i], C::OFF_Q, r);
                    if (p.have_ds) scale(C::TM_DK, sWt[i], C::OFF_K, e);
                    sR[i] = r;
                    sE[i] = e;
                    ok = wwait(&m->dv_full, ph);
                    if (ok) {
                        tc_fence_after();
                        if (p.have_ds) scale(C::TM_DV, sWt[i], -1, none);
                        tmem_st_wait();
                        tc_fence_before();
                        mbar_arrive(&m->scaled);
                    }
                }
            }
            // ------------------------------------------------------------ results
            if (ok) ok = wwait(&m->out_full, ph);
            if (ok) {
                tc_fence_after();
                auto store = [&](uint32_t col, __nv_bfloat16 *out, int c0, int c1) {
#pragma unroll 1
                    for (int cc = c0; cc < c1; ++cc) {
                        uint32_t a[32];
                        tmem_ld32(tmem + col + 32 * cc + lanes, a);
                        tmem_ld_wait();
                        if (i < nv) {
                            uint4 *dst = reinterpret_cast<uint4 *>(out + ((size_t)(row0 + i) * p.H + h) * D + 32 * cc);
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                dst[y] = make_uint4(
                                    pack_bf16x2(__uint_as_float(a[8 * y]), __uint_as_float(a[8 * y + 1])),
                                    pack_bf16x2(__uint_as_float(a[8 * y + 2]), __uint_as_float(a[8 * y + 3])),
                                    pack_bf16x2(__uint_as_float(a[8 * y + 4]), __uint_as_float(a[8 * y + 5])),
                                    pack_bf16x2(__uint_as_float(a[8 * y + 6]), __uint_as_float(a[8 * y + 7])));
                        }
                    }
                };
                if (warp < 6) {
                    store(C::TM_DK, p.dk, 0, D / 32);
                    store(C::TM_DV, p.dv, 0, D / 64);
                } else {
                    store(C::TM_DQ, p.dq, 0, D / 32);
                    store(C::TM_DV, p.dv, D / 64, D / 32);
                }
                tc_fence_before();
            }
        }
        if (!ok) fail();
        // TMEM, the decays and the sums are free for the next block
        if (__syncthreads_or(!ok)) {
            ok = false;
            break;
        }
        tc_fence_after();
    }
    if (tid == 0 && !ok) {  // loads that are still in flight land before the CTA ends
        mbar_wait(&m->full_qk, load_phase, nullptr, tlimit);
        mbar_wait(&m->full_vo, load_phase, nullptr, tlimit);
        mbar_wait(&m->full_ss, load_phase, nullptr, tlimit);
    }
    if (warp == 1 && lane == 0) {  // every issued MMA has finished before TMEM is freed
        mma_commit(&m->done);
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
