// The state scan of gated lightning attention on the tensor cores (bf16 inputs).
//
//   forward   X = state at a block's start,        X <- e^{G_C} X + sum_j k_j (e^{G_C - G_j} v_j)^T
//   reverse   X = state gradient at its end,       X <- e^{G_C} X + sum_i q_i (e^{G_i} do_i)^T
//
// over blocks of C = 128 tokens; the bf16 value of X before each update goes to a snapshot
// per block, from which the block kernels then run independently of each other.
//
// One CTA per (segment, head, 64-column slice of the state).  Per block the tile of the left
// factor (128 x D) and the slice of the right one (128 x 64) arrive by TMA; six warps scale
// the slice's rows by their decays and split every product into three bf16 numbers whose sum
// is the fp32 product to 2^-26 (one bf16 alone would round the state by 2^-9 in every step);
// one thread issues a single product [D x 128] [128 x 192] of the tile with the three parts
// side by side (one read of the left factor from shared memory instead of three), and the
// epilogue adds the three accumulators to the fp32 state in its registers.
//
// The tensor work (3 x 2 D^2 flops per token) is below its HBM time: 4 D bytes read (the left
// tile is read by D / 64 CTAs, mostly from L2) and 2 D^2 / 128 bytes of snapshot written per
// token and head.
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
    __nv_bfloat16 *snap;        // [blocks][H][D][D] or nullptr
    const __nv_bfloat16 *other; // reverse: the forward snapshots, or nullptr
    float *through;             // reverse: [blocks][H][4 D / 64] parts of e^{G_C} <X, state>
    int H;
    unsigned long long timeout_ns;
    GatedTable tab;
};

template <int D>
struct GatedStateCfg {
    static constexpr int C = 128;
    static constexpr int NVS = D / 64;              // column slices (CTAs) per (segment, head)
    static constexpr int DB = D / 64;               // 64-column boxes of the left tile
    static constexpr int BOX = C * 128;             // 128 rows x 128 B
    static constexpr int STAGE = (DB + 3) * BOX;    // left tile, then the slice and its two lower parts
    static constexpr int LOADED = (DB + 1) * BOX;
    static constexpr int NST = 2;
    static constexpr int SCALERS = 6;               // warps (12 in all: 168 registers a thread)
    static constexpr int OFF_W = NST * STAGE;       // decays, 128 floats per scaling warp
    static constexpr int OFF_MISC = OFF_W + SCALERS * C * 4;
    static constexpr int SMEM_USED = 1024 + OFF_MISC + 1024;
    // above half of the SM's shared memory: two CTAs of one SM would wait for TMEM
    static constexpr int SMEM_BYTES = SMEM_USED < 120 * 1024 ? 120 * 1024 : SMEM_USED;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
    static constexpr int TMEM_COLS = 512;           // two accumulators of 192 columns
    static constexpr int ACC = 256;                 // columns from one accumulator to the other
    static constexpr int GROUP = 128;               // epilogue threads
    static constexpr int THREADS = 64 + GROUP + 32 * SCALERS;
    static constexpr uint32_t ID = idesc_bf16_f32(D, 192, 1, 1);
};

struct GatedStateMisc {
    uint64_t full[2], ready[2], empty[2];  // tiles landed, scaled, released
    uint64_t acc_full[2], acc_free[2];
    uint64_t done;
    uint32_t tmem_base;
    int abort_flag;
};

// The log-decays of tokens 4 * lane .. 4 * lane + 3 of a block (0 behind the sequence).
__device__ __forceinline__ void load_gates4(float (&x)[4], const __nv_bfloat16 *__restrict__ g, int row0,
                                            int nv, int H, int h) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = 4 * lane + e;
        x[e] = g != nullptr && i < nv ? clamp_gate(__bfloat162float(g[(size_t)(row0 + i) * H + h])) : 0.f;
    }
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

// One 16-byte chunk of eight bf16 values scaled by w, as three bf16 parts.  `keep` false
// gives zeros whatever the chunk holds.
__device__ __forceinline__ void split3(const uint4 &raw, float w, bool keep, uint4 &p0, uint4 &p1, uint4 &p2) {
    const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t out[3][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float lo = keep ? w * __uint_as_float(in[e] << 16) : 0.f;
        float hi = keep ? w * __uint_as_float(in[e] & 0xffff0000u) : 0.f;
#pragma unroll
        for (int part = 0; part < 3; ++part) {
            const uint32_t pk = pack_bf16x2(lo, hi);
            out[part][e] = pk;
            lo -= __uint_as_float(pk << 16);
            hi -= __uint_as_float(pk & 0xffff0000u);
        }
    }
    p0 = make_uint4(out[0][0], out[0][1], out[0][2], out[0][3]);
    p1 = make_uint4(out[1][0], out[1][1], out[1][2], out[1][3]);
    p2 = make_uint4(out[2][0], out[2][1], out[2][2], out[2][3]);
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
__device__ __forceinline__ void st_shared_u4(uint32_t addr, const uint4 &v) {
    st_shared_v4(addr, v.x, v.y, v.z, v.w);
}

template <int D, bool REV>
__global__ void __launch_bounds__(GatedStateCfg<D>::THREADS, 1)
    gated_state_tc_kernel(const __grid_constant__ GatedStateParams p) {
    using C = GatedStateCfg<D>;
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
    const uint64_t tlimit = p.timeout_ns;
    volatile int *abort_flag = &m->abort_flag;
    // the t-th block that the scan visits, and its tokens
    auto block_of = [&](int t) { return REV ? b0 + nb - 1 - t : b0 + t; };
    auto rows_of = [&](int blk) { return min(C::C, len - blk * C::C); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m->full[i], 1);
            mbar_init(&m->ready[i], 32 * C::SCALERS);
            mbar_init(&m->empty[i], 1);
            mbar_init(&m->acc_full[i], 1);
            mbar_init(&m->acc_free[i], C::GROUP);
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
    auto fail = [&]() {
        *abort_flag = 1;
        record_fault(DEV_TIMEOUT);
    };
    auto wwait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, tlimit)) != 0;
    };
    // Every ring has two slots: use t of a slot is its phase t / 2, and a slot is refilled
    // only after its release of use t - 2, so that each wait below sees the phase it means.
    auto stage = [&](int t) { return sbase + (uint32_t)((t & 1) * C::STAGE); };

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer
        if (lane == 0) {
            int issued = 0;
            for (int t = 0; t < nb; ++t) {
                if (!mbar_wait(&m->empty[t & 1], (uint32_t)(((t >> 1) & 1) ^ 1), abort_flag, tlimit)) {
                    fail();
                    break;
                }
                mbar_arrive_expect_tx(&m->full[t & 1], (uint32_t)C::LOADED);
                const int row = start + block_of(t) * C::C, col = h * D;
#pragma unroll
                for (int d = 0; d < C::DB; ++d)
                    tma_load_2d(stage(t) + d * C::BOX, &p.tmap_a, col + 64 * d, row, &m->full[t & 1]);
                tma_load_2d(stage(t) + C::DB * C::BOX, &p.tmap_b, col + 64 * vs, row, &m->full[t & 1]);
                ++issued;
            }
            for (int t = max(0, issued - 2); t < issued; ++t)
                mbar_wait(&m->full[t & 1], (uint32_t)((t >> 1) & 1), nullptr, tlimit);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        bool ok = true;
        for (int t = 0; t < nb; ++t) {
            if (!wwait(&m->full[t & 1], (uint32_t)((t >> 1) & 1)) ||
                !wwait(&m->ready[t & 1], (uint32_t)((t >> 1) & 1)) ||
                (t >= 2 && !wwait(&m->acc_free[t & 1], (uint32_t)(((t - 2) >> 1) & 1)))) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (lane == 0) {  // [dims][3 x 64 columns] = A^T [part 0 | part 1 | part 2]
                const uint64_t ad = desc_mnmajor_sw128(stage(t), C::BOX);
                const uint64_t bd = desc_mnmajor_sw128(stage(t) + C::DB * C::BOX, C::BOX);
#pragma unroll
                for (int ks = 0; ks < C::C / 16; ++ks)
                    mma_bf16_ss(tmem + C::ACC * (t & 1), desc_add(ad, ks * 2048), desc_add(bd, ks * 2048),
                                C::ID, ks > 0 ? 1u : 0u);
                mma_commit(&m->empty[t & 1]);
                mma_commit(&m->acc_full[t & 1]);
            }
            __syncwarp();
        }
        if (!ok) fail();
        if (lane == 0) {  // every issued MMA has finished before TMEM is freed
            mma_commit(&m->done);
            mbar_wait(&m->done, 0u, nullptr, tlimit);
        }
        __syncwarp();
    } else if (warp < 6) {
        // ---------------------------------------------------------------- epilogue: the state
        const int q = warp & 3;
        // row i of the accumulators: lane i for M = 128; lanes 0..15 of each 32-lane
        // quadrant for M = 64
        const int i = D == 128 ? 32 * q + lane : 16 * q + lane;
        const bool i_ok = D == 128 || lane < 16;
        const uint32_t lane_base = (uint32_t)(32 * q) << 16;
        float X[64];  // X[i][64 vs .. 64 vs + 63]
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
        const size_t first = (size_t)p.tab.first_block(rank);
        float gate[4], sums[4], total = 0.f;
        if (nb > 0) load_gates4(gate, p.g, start + block_of(0) * C::C, rows_of(block_of(0)), p.H, h);
        bool ok = true;
        for (int t = 0; t < nb; ++t) {
            const int blk = block_of(t);
            const size_t at = (first + blk) * p.H + h;
            const float G = prefix_gates4(gate, sums), decay = expf(G);
            total += G;
            if (t + 1 < nb)
                load_gates4(gate, p.g, start + block_of(t + 1) * C::C, rows_of(block_of(t + 1)), p.H, h);
            if (REV && p.through != nullptr) {
                // part of e^{G_C} <X, state at the block's start>: this warp's rows and columns
                float f = 0.f;
                if (i_ok) {
                    const uint4 *o = reinterpret_cast<const uint4 *>(p.other + (at * D + i) * D + 64 * vs);
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const uint4 w = o[x];
                        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            f = fmaf(__uint_as_float(in[e] << 16), X[8 * x + 2 * e], f);
                            f = fmaf(__uint_as_float(in[e] & 0xffff0000u), X[8 * x + 2 * e + 1], f);
                        }
                    }
                }
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) f += __shfl_xor_sync(0xffffffffu, f, off);
                if (lane == 0) p.through[at * (4 * C::NVS) + 4 * vs + q] = decay * f;
            }
            if (p.snap != nullptr && i_ok) {
                uint4 *d = reinterpret_cast<uint4 *>(p.snap + (at * D + i) * D + 64 * vs);
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    d[x] = make_uint4(pack_bf16x2(X[8 * x], X[8 * x + 1]), pack_bf16x2(X[8 * x + 2], X[8 * x + 3]),
                                      pack_bf16x2(X[8 * x + 4], X[8 * x + 5]),
                                      pack_bf16x2(X[8 * x + 6], X[8 * x + 7]));
            }
            if (!wwait(&m->acc_full[t & 1], (uint32_t)((t >> 1) & 1))) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t tA = tmem + C::ACC * (t & 1) + lane_base;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t a[32];
                // the smallest part first
                tmem_ld32(tA + 128 + 32 * half, a);
                tmem_ld_wait();
                float lo[32];
#pragma unroll
                for (int x = 0; x < 32; ++x) lo[x] = __uint_as_float(a[x]);
                tmem_ld32(tA + 64 + 32 * half, a);
                tmem_ld_wait();
#pragma unroll
                for (int x = 0; x < 32; ++x) lo[x] += __uint_as_float(a[x]);
                tmem_ld32(tA + 32 * half, a);
                tmem_ld_wait();
                if (half == 1) {
                    tc_fence_before();
                    mbar_arrive(&m->acc_free[t & 1]);
                }
#pragma unroll
                for (int x = 0; x < 32; ++x)
                    X[32 * half + x] = fmaf(decay, X[32 * half + x], lo[x] + __uint_as_float(a[x]));
            }
        }
        float *to = nullptr;
        if (p.seg_out != nullptr)
            to = p.seg_out + ((size_t)sg * p.H + h) * D * D;
        else if (p.fin != nullptr && s == (REV ? 0 : p.tab.num_segs(rank) - 1))
            to = p.fin + ((size_t)sid * p.H + h) * D * D;
        if (ok && to != nullptr && i_ok) {
            float4 *d4 = reinterpret_cast<float4 *>(to + (size_t)i * D + 64 * vs);
#pragma unroll
            for (int x = 0; x < 16; ++x) d4[x] = make_float4(X[4 * x], X[4 * x + 1], X[4 * x + 2], X[4 * x + 3]);
        }
        if (ok && p.seg_out != nullptr && vs == 0 && q == 0 && lane == 0) p.seg_total[(size_t)sg * p.H + h] = total;
        if (!ok) fail();
    } else {
        // ---------------------------------------------------------------- scaling warps
        const int w8 = warp - 6;
        float *sw = reinterpret_cast<float *>(smem + C::OFF_W) + w8 * C::C;  // this warp's own copy
        float gate[4], sums[4];
        if (nb > 0) load_gates4(gate, p.g, start + block_of(0) * C::C, rows_of(block_of(0)), p.H, h);
        bool ok = true;
        for (int t = 0; t < nb; ++t) {
            const int nv = rows_of(block_of(t));
            if (REV)
                prefix_gates4(gate, sums);
            else
                suffix_gates4(gate, sums);
            if (t + 1 < nb)
                load_gates4(gate, p.g, start + block_of(t + 1) * C::C, rows_of(block_of(t + 1)), p.H, h);
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 4; ++e) sw[4 * lane + e] = expf(sums[e]);
            __syncwarp();
            if (!wwait(&m->full[t & 1], (uint32_t)((t >> 1) & 1))) {
                ok = false;
                break;
            }
            const uint32_t b = stage(t) + C::DB * C::BOX;
            // chunk c of row r lies in one of the row's eight 16-byte places, whichever the
            // swizzle says; all eight are scaled alike
#pragma unroll 2
            for (int c = w8 * 32 + lane; c < C::C * 8; c += 32 * C::SCALERS) {
                const int r = c >> 3;
                uint4 p0, p1, p2;
                split3(ld_shared_v4(b + c * 16), sw[r], r < nv, p0, p1, p2);
                st_shared_u4(b + c * 16, p0);
                st_shared_u4(b + C::BOX + c * 16, p1);
                st_shared_u4(b + 2 * C::BOX + c * 16, p2);
            }
            if (nv < C::C)  // rows of another sequence: 0 times what they hold could be a NaN
                for (int d = 0; d < C::DB; ++d)
                    for (int c = nv * 8 + w8 * 32 + lane; c < C::C * 8; c += 32 * C::SCALERS)
                        st_shared_v4(stage(t) + d * C::BOX + c * 16, 0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            mbar_arrive(&m->ready[t & 1]);
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
