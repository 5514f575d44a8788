// liblightning.so: the C ABI declared in include/lightning_attention.h.
//
// Host side only: argument validation, the sequence table, TMA tensor maps and
// kernel launches.  Every step of the computation runs in the kernels of
// prefill_pair.cuh and prefill_tc.cuh (bf16, tcgen05), prefill_simt.cuh (fp32),
// chunk_state.cuh, decode.cuh and the gated*.cuh files.
#include <algorithm>
#include <atomic>
#include <cstdio>
#include <cstring>
#include <type_traits>

#include "chunk_state.cuh"
#include "decode.cuh"
#include "gated.cuh"
#include "gated_backward_tc.cuh"
#include "gated_prefill_tc.cuh"
#include "gated_state_tc.cuh"
#include "prefill_simt.cuh"
#include "prefill_pair.cuh"
#include "prefill_tc.cuh"
#include "selftest.cuh"

namespace {

using la::PrefillTcParams;
using la::SeqTable;

constexpr int kSMs = 148;
constexpr unsigned long long kWaitLimitNs = 1000ull * 1000ull * 1000ull;  // 1 s per wait

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// cuTensorMapEncodeTiled, fetched through the runtime so that the library does
// not link libcuda directly.
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// (Threads that come first together each ask, and get the same answer.)
EncodeTiledFn encode_fn() {
    static std::atomic<EncodeTiledFn> known{nullptr};
    EncodeTiledFn fn = known.load(std::memory_order_acquire);
    if (fn != nullptr) return fn;
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
        fn = reinterpret_cast<EncodeTiledFn>(p);
        known.store(fn, std::memory_order_release);
    }
    return fn;
}

// [T][H*D] bf16 viewed as a 2-D tensor; boxes of 64 columns x beta rows, 128-B swizzle.
bool make_map(CUtensorMap *map, const void *base, long long T, int H, int D, int beta) {
    EncodeTiledFn fn = encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[2] = {(cuuint64_t)H * D, (cuuint64_t)T};
    cuuint64_t strides[1] = {(cuuint64_t)H * D * 2};
    cuuint32_t box[2] = {64, (cuuint32_t)beta};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

// The sequence table of a call: B equal sequences of N tokens, or the packed
// boundaries cu_seqlens (host array, validated here), ordered longest first so
// that the block scheduler starts the longest chains first (equal ones in their order).
la_status build_seq_table(int B, int N, const int32_t *cu_seqlens, int num_seqs, SeqTable &seqs,
                          long long &T, int &S) {
    std::memset(&seqs, 0, sizeof seqs);
    T = 0;
    S = 0;
    if (cu_seqlens != nullptr) {
        if (B != 1) return LA_ERR_INVALID_ARG;
        if (num_seqs < 1) return LA_ERR_INVALID_ARG;
        if (num_seqs > LA_MAX_VARLEN_SEQS) return LA_ERR_UNSUPPORTED;
        if (cu_seqlens[0] != 0 || cu_seqlens[num_seqs] != N) return LA_ERR_INVALID_ARG;
        for (int s = 0; s < num_seqs; ++s)
            if (cu_seqlens[s + 1] < cu_seqlens[s]) return LA_ERR_INVALID_ARG;
        S = num_seqs;
        T = N;
        // (no allocation, which could throw across the C boundary)
        int order[LA_MAX_VARLEN_SEQS];
        for (int s = 0; s < S; ++s) order[s] = s;
        std::sort(order, order + S, [&](int a, int b) {
            const int la = cu_seqlens[a + 1] - cu_seqlens[a], lb = cu_seqlens[b + 1] - cu_seqlens[b];
            return la != lb ? la > lb : a < b;
        });
        seqs.varlen = 1;
        for (int r = 0; r < S; ++r) {
            const int s = order[r];
            seqs.seq_start[r] = cu_seqlens[s];
            seqs.seq_len[r] = cu_seqlens[s + 1] - cu_seqlens[s];
            seqs.seq_id[r] = s;
        }
    } else {
        S = B;
        T = (long long)B * N;
        seqs.varlen = 0;
        seqs.N = N;
    }
    return LA_OK;
}

template <int BETA, int D>
la_status launch_tc(const PrefillTcParams &p, int units, cudaStream_t stream) {
    using C = la::TcCfg<BETA, D>;
    auto kern = la::prefill_tc_kernel<BETA, D>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) !=
        cudaSuccess)
        return LA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)units);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C::NVS;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

la_status launch_pair(const la::PrefillPairParams &p, int pairs, cudaStream_t stream) {
    using C = la::PairCfg;
    auto kern = la::prefill_pair_kernel;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) !=
        cudaSuccess)
        return LA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

template <int BETA, int D>
la_status launch_simt(const float *q, const float *k, const float *v, float *o, float *state,
                      const float *state_in, int H, int rmsnorm, const SeqTable &seqs, int S,
                      cudaStream_t stream) {
    using C = la::SimtCfg<BETA, D>;
    auto kern = la::prefill_simt_kernel<BETA, D>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) !=
        cudaSuccess)
        return LA_ERR_CUDA;
    kern<<<S * H, C::THREADS, C::SMEM_BYTES, stream>>>(q, k, v, o, state, state_in, H, rmsnorm, seqs);
    return cudaGetLastError() == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}


// ------------------------------------------------------------------ gated operators
using la::GatedTable;

// A row looks for its slot among the rows before it: at this many, 128 KB of them on average,
// what the state of a row at D = 128 takes too.
constexpr int LA_MAX_SLOT_ROWS = 65536;

struct GatedPlan {
    GatedTable tab;
    bool segmented;
    bool simt;                     // on the CUDA cores: fp32, and backward passes of short sequences
    bool joined;                   // fp32: segments of one block, whose start states are the snapshots
    int longest;                   // blocks of the longest sequence
    // prefill: the sequences of one token, which are decode steps and not in the table (one
    // would hold a whole CTA per slice for one row)
    la::OneTokenTable one;
    int ones;
    // workspace offsets (bytes): state snapshots of both directions, the parts of <dS, S>,
    // segment states, their decays
    size_t snap, dsnap, through, seg_state, seg_total, bytes;
};

constexpr int kShortTokens = 16, kShortRows = 2 * kSMs;

// The table and the workspace of a call.  A state scan runs one CTA per (segment, head,
// slice), one block after the other.  Cutting sequences into segments shortens the longest
// chain, at the price of a scan before (the segments' own end states, a second read of the
// scan's inputs) and a kernel that joins them.  Segments as long as fill the GPU once, at
// least 4 blocks; taken where they pay: beside two scans of `seg` blocks there is a second
// scan's start and the joining, about the time of 12 blocks (measured: 1.2 to 1.6 us a block,
// 8 us a start, 6 us the joining).
la_status plan_gated(int B, int H, int N, int D, const int32_t *cu_seqlens, int num_seqs, unsigned flags,
                     bool backward, GatedPlan &pl, long long &T) {
    int S = 0;
    GatedTable &t = pl.tab;
    if (la_status st = build_seq_table(B, N, cu_seqlens, num_seqs, t.seqs, T, S); st != LA_OK) return st;
    // tensor cores: 128-token blocks, snapshots in two bf16 parts (of the backward pass alone: the
    // prefill kernel keeps its state on chip); CUDA cores: 64-token blocks, fp32 snapshots
    // The backward pass of a few short sequences runs on the CUDA cores whatever the type.  It is
    // one or two kernels instead of three: 16 tokens of 64 heads take 10 us of GPU time and not 12
    // at D = 64 (with states 21 and not 23), 14 and 14 (37 and 31) at D = 128; of 256 (sequence,
    // head) pairs 13 and not 19 (29 and 41), 27 and 25 (78 and 79).  And scores stay fp32: P of one
    // token is a single number, whose bf16 rounding shifts a whole row of dk or dv (1.3 times the
    // result's own rounding in the median, 3 times at most; here 1.0).
    const int most = t.seqs.varlen ? (S > 0 ? t.seqs.seq_len[0] : 0) : N;
    pl.simt = (flags & LA_BF16) == 0 || (backward && most <= kShortTokens && (long long)S * H <= kShortRows);
    const bool tc = !pl.simt;
    const int C = tc ? 128 : la::GatedSimt::C, slices = tc ? D / 64 : D / la::GatedSimt::VS;
    const int resident = kSMs, min_seg = 4;
    pl.ones = pl.one.identity = 0;
    if (!backward) {
        if (t.seqs.varlen) {
            int w = 0;
            for (int r = 0; r < S; ++r) {
                if (t.seqs.seq_len[r] == 1) {
                    pl.one.row[pl.ones] = t.seqs.seq_start[r];
                    pl.one.sid[pl.ones++] = t.seqs.seq_id[r];
                } else {
                    t.seqs.seq_start[w] = t.seqs.seq_start[r];
                    t.seqs.seq_len[w] = t.seqs.seq_len[r];
                    t.seqs.seq_id[w++] = t.seqs.seq_id[r];
                }
            }
            S = w;
        } else if (N == 1) {
            pl.one.identity = 1;
            pl.ones = S;
            S = 0;
        }
    }
    t.S = S;
    t.C = C;
    long long blocks = 0;
    pl.longest = 0;
    auto blocks_of = [&](int len) { return (int)(((long long)len + C - 1) / C); };
    for (int r = 0; r < (t.seqs.varlen ? S : std::min(S, 1)); ++r) {
        const int nb = blocks_of(t.seqs.varlen ? t.seqs.seq_len[r] : N);
        pl.longest = std::max(pl.longest, nb);
        blocks += t.seqs.varlen ? nb : (long long)nb * S;
    }
    // the shortest segments of which no more than `resident` CTAs come, else of which every CTA
    // has about the same share
    auto segments = [&](long long seg) {
        if (!t.seqs.varlen) return (long long)S * std::max(1ll, (pl.longest + seg - 1) / seg);
        long long n = 0;
        for (int r = 0; r < S; ++r) n += std::max(1ll, (blocks_of(t.seqs.seq_len[r]) + seg - 1) / seg);
        return n;
    };
    const long long room = resident / ((long long)H * slices);
    long long seg = std::max<long long>(min_seg, (blocks * H * slices + resident - 1) / resident);
    if (S <= room) {
        long long lo = seg, hi = std::max<long long>(seg, pl.longest);  // segments(hi) <= room
        while (lo < hi) {
            const long long mid = (lo + hi) / 2;
            if (segments(mid) <= room)
                hi = mid;
            else
                lo = mid + 1;
        }
        seg = lo;
    }
    pl.segmented = pl.longest > 2 * seg + 12;
    // fp32: a block's snapshot is the start state of a segment of one block, so that with such
    // segments the scan is one block long and joining them is all the rest.  Taken where the
    // scan has SMs to spare (4 heads of 1000 tokens, D = 64, backward: 45 us and not 108; 64
    // heads of 256, D = 128: 176 and not 159), the segments' own states, written and read once
    // more, stay in L2, and joining (0.15 us a block) takes less than the chain (3 us a block;
    // 1 head of 32768 tokens, D = 64: 243 us and not 184).  A forward call of fewer than eight
    // blocks would wait for the host's third launch instead (2 heads of 256: 16 us of GPU time
    // and not 22, but 31 and not 25 from call to call).
    pl.joined = !tc && pl.longest >= (backward ? 4 : 8) && S <= room && blocks * H * D * D * 4 <= (32ll << 20) &&
                pl.longest + 20 < 20 * (pl.segmented ? 2 * seg + 3 : pl.longest);
    if (pl.joined) pl.segmented = true, seg = 1;
    t.seg_blocks = pl.segmented ? (int)seg : std::max(1, pl.longest);
    long long nblk = 0, nseg = 0;
    if (t.seqs.varlen) {
        for (int r = 0; r < S; ++r) {
            const int nb = blocks_of(t.seqs.seq_len[r]);
            t.block0[r] = (int)nblk;
            t.seg0[r] = (int)nseg;
            nblk += nb;
            nseg += std::max(1, (nb + t.seg_blocks - 1) / t.seg_blocks);
        }
        t.block0[S] = (int)nblk;
        t.seg0[S] = (int)nseg;
        t.blocks_per_seq = t.segs_per_seq = 0;
    } else {
        t.blocks_per_seq = pl.longest;
        t.segs_per_seq = std::max(1, (pl.longest + t.seg_blocks - 1) / t.seg_blocks);
        nblk = (long long)S * t.blocks_per_seq;
        nseg = (long long)S * t.segs_per_seq;
    }
    // (the snapshots' rows, two parts of nblk * H * D, are coordinates of a tensor map)
    if (T >= (1ll << 31) || 2 * nblk * H * D >= (1ll << 31) || nseg * H * slices >= (1ll << 31) ||
        (long long)pl.ones * H >= (1ll << 31))
        return LA_ERR_UNSUPPORTED;
    t.blocks = (int)nblk;
    t.segs = (int)nseg;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t o = at;
        at += (n + 255) & ~(size_t)255;
        return o;
    };
    const size_t state = (size_t)D * D * 4, shot = state;
    // (joined: the table has the sequences without blocks, which count as a segment, last)
    const bool own = !tc && backward && pl.longest <= 1;  // the call's own states serve
    const size_t shots = own ? 0 : (size_t)(pl.joined ? nseg : nblk) * H * shot;
    pl.snap = take(tc && !backward ? 0 : shots);
    pl.dsnap = take(backward ? shots : 0);
    pl.through = take(tc && backward ? (size_t)nblk * H * 8 * slices * 4 : 0);
    pl.seg_state = take(pl.segmented && !pl.joined ? (size_t)nseg * H * state : 0);
    pl.seg_total = take(pl.segmented ? (size_t)nseg * H * 4 : 0);
    pl.bytes = at;
    return LA_OK;
}

la_status launched() { return cudaGetLastError() == cudaSuccess ? LA_OK : LA_ERR_CUDA; }

// Launch; `behind`: a later kernel of the same call, whose CTAs may start before the kernel
// before it has ended (they wait for its results themselves, see gated.cuh).
template <typename T>
struct as_given {
    using type = T;
};
template <typename... P>
la_status launch_behind(bool behind, void (*kern)(P...), dim3 grid, int threads, int smem, cudaStream_t stream,
                        const typename as_given<P>::type &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = behind ? 1 : 0;
    // (by address: the tables are 20 KB)
    void *at[] = {const_cast<void *>(static_cast<const void *>(&args))...};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(kern), at) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

// The sequences of one token of a prefill call.
template <int D, typename E>
la_status gated_rows(const void *q, const void *k, const void *v, const void *g, void *o, const float *state_in,
                     float *state_out, int H, const GatedPlan &pl, cudaStream_t stream) {
    la::gated_rows_kernel<D, E><<<(unsigned)(pl.ones * H), 256, 0, stream>>>(
        static_cast<const E *>(q), static_cast<const E *>(k), static_cast<const E *>(v), static_cast<const E *>(g),
        static_cast<E *>(o), state_in, state_out, H, pl.one);
    return launched();
}

// State scan of one direction: snapshots per block, the final state where wanted.
template <int D, bool REV, typename E>
la_status gated_states_simt(const E *a, const E *b, const E *g, const float *initial, float *snap,
                            float *fin, int H, const GatedPlan &pl, uint8_t *ws, bool behind, cudaStream_t stream) {
    auto kern = la::gated_state_simt_kernel<D, REV, E>;
    constexpr int smem = la::GatedStateSimt<D>::SMEM_BYTES;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return LA_ERR_CUDA;
    const unsigned grid = (unsigned)(pl.tab.segs * H * (D / la::GatedSimt::VS));
    float *seg_state = nullptr, *seg_total = nullptr;
    if (pl.segmented) {
        seg_state = pl.joined ? snap : reinterpret_cast<float *>(ws + pl.seg_state);
        seg_total = reinterpret_cast<float *>(ws + pl.seg_total);
        const float *none = nullptr;
        if (la_status st = launch_behind(behind, kern, dim3(grid), la::GatedStateSimt<D>::THREADS, smem, stream, a, b, g,
                                         none, none, seg_state, seg_total, nullptr, nullptr, H, pl.tab);
            st != LA_OK)
            return st;
        la_status st = launch_behind(true, la::gated_prefix_kernel, dim3((unsigned)(pl.tab.S * H), D * D / 1024), 256,
                                     0, stream, reinterpret_cast<float4 *>(seg_state), seg_total,
                                     reinterpret_cast<const float4 *>(initial),
                                     pl.joined ? reinterpret_cast<float4 *>(fin) : nullptr, H, D * D / 4, REV ? 1 : 0,
                                     pl.tab);
        if (st != LA_OK || pl.joined) return st;
    }
    // (not behind the joining kernel: CTAs that start while SMs are still taken end up two to an
    // SM beside idle ones; 32768 tokens of one head, D = 64, forward: 87 us, not 78)
    return launch_behind(behind && !pl.segmented, kern, dim3(grid), la::GatedStateSimt<D>::THREADS, smem, stream, a, b, g,
                         initial, seg_state, nullptr, nullptr, snap, fin, H, pl.tab);
}

template <int D>
la_status gated_prefill_simt(const float *q, const float *k, const float *v, const float *g, float *o,
                             const float *state_in, float *state_out, int H, const GatedPlan &pl, uint8_t *ws,
                             cudaStream_t stream) {
    float *snap = nullptr;
    if (pl.longest > 1 || state_in != nullptr) snap = reinterpret_cast<float *>(ws + pl.snap);
    if (snap != nullptr || state_out != nullptr)
        if (la_status st = gated_states_simt<D, false>(k, v, g, state_in, snap, state_out, H, pl, ws, false, stream);
            st != LA_OK)
            return st;
    if (pl.tab.blocks == 0) return LA_OK;  // beside sequences of one token only empty ones
    auto kern = la::gated_prefill_simt_kernel<D>;
    constexpr int smem = la::GatedSimtTiles<D>::FWD_BYTES;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return LA_ERR_CUDA;
    return launch_behind(snap != nullptr || state_out != nullptr, kern, dim3((unsigned)(pl.tab.blocks * H)),
                         la::GatedSimt::THREADS, smem, stream, q, k, v, g, o, snap, H, pl.tab);
}

template <int D, typename E>
la_status gated_backward_simt(const void *q_, const void *k_, const void *v_, const void *g_, const void *dout_, void *dq,
                              void *dk, void *dv, void *dg, const float *state_in, const float *d_state,
                              float *d_state_in, int H, const GatedPlan &pl, uint8_t *ws, cudaStream_t stream) {
    const E *q = static_cast<const E *>(q_), *k = static_cast<const E *>(k_), *v = static_cast<const E *>(v_),
            *g = static_cast<const E *>(g_), *dout = static_cast<const E *>(dout_);
    auto kern = la::gated_backward_simt_kernel<D, E>;
    constexpr int smem = la::GatedSimtTiles<D>::BWD_BYTES;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return LA_ERR_CUDA;
    auto blocks = [&](bool behind, const float *snap, const float *dsnap, int by_seq) {
        return launch_behind(behind, kern, dim3((unsigned)(pl.tab.blocks * H)), la::GatedSimt::THREADS, smem, stream, q,
                             k, v, g, dout, static_cast<E *>(dq), static_cast<E *>(dk), static_cast<E *>(dv),
                             static_cast<E *>(dg), snap, dsnap, by_seq, H, pl.tab);
    };
    if (pl.longest <= 1) {
        // no block but the first: its states are the call's.  (d_state_in may be d_state: last.)
        if (la_status st = blocks(false, state_in, d_state, 1); st != LA_OK || d_state_in == nullptr) return st;
        return gated_states_simt<D, true>(q, dout, g, d_state, nullptr, d_state_in, H, pl, ws, true, stream);
    }
    float *snap = reinterpret_cast<float *>(ws + pl.snap), *dsnap = reinterpret_cast<float *>(ws + pl.dsnap);
    if constexpr (std::is_same_v<E, float>) {
        if (la_status st = gated_states_simt<D, false>(k, v, g, state_in, snap, nullptr, H, pl, ws, false, stream);
            st != LA_OK)
            return st;
        if (la_status st = gated_states_simt<D, true>(q, dout, g, d_state, dsnap, d_state_in, H, pl, ws, true, stream);
            st != LA_OK)
            return st;
        return blocks(true, snap, dsnap, 0);
    }
    return LA_ERR_UNSUPPORTED;  // bf16 comes here with single blocks alone
}

// The tensor-core state scan of one direction (bf16): a = k, b = v, or reversed a = q, b = do.
// The kernels whose warpgroups trade registers (setmaxnreg) have to start with what the shares
// add up to, or a group would wait for registers that nobody gives back.
// The registers are a property of the build, so they are asked for until the first answer.
template <typename K>
bool starts_with(K kern, int registers, std::atomic<bool> &known) {
    if (known.load(std::memory_order_relaxed)) return true;
    cudaFuncAttributes at;
    if (cudaFuncGetAttributes(&at, kern) != cudaSuccess || at.numRegs < registers) return false;
    known.store(true, std::memory_order_relaxed);
    return true;
}

template <int D, bool REV>
la_status launch_gated_states(const la::GatedStateParams &p, bool behind, cudaStream_t stream) {
    using C = la::GatedStateCfg<D, REV>;
    auto kern = la::gated_state_tc_kernel<D, REV>;
    static std::atomic<bool> fits{false};
    if (!starts_with(kern, C::R_LAUNCH, fits)) return LA_ERR_CUDA;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess)
        return LA_ERR_CUDA;
    return launch_behind(behind, kern, dim3((unsigned)(p.tab.segs * p.H * C::NVS)), C::THREADS, C::SMEM_BYTES, stream, p);
}

template <int D>
bool fill_gated_states(la::GatedStateParams &p, const void *a, const void *b, const void *g, int H, long long T,
                       const GatedPlan &pl) {
    std::memset(&p, 0, sizeof p);
    p.g = static_cast<const __nv_bfloat16 *>(g);
    p.H = H;
    p.timeout_ns = kWaitLimitNs;
    p.tab = pl.tab;
    return make_map(&p.tmap_a, a, T, H, D, 128) && make_map(&p.tmap_b, b, T, H, D, 128);
}

// The start states of a segmented call's segments (in place of their own end states).
template <int D, bool REV>
la_status gated_seg_states_tc(la::GatedStateParams p, const float *initial, const GatedPlan &pl, uint8_t *ws,
                              bool behind, cudaStream_t stream, float *&seg_in) {
    p.seg_out = seg_in = reinterpret_cast<float *>(ws + pl.seg_state);
    p.seg_total = reinterpret_cast<float *>(ws + pl.seg_total);
    if (la_status st = launch_gated_states<D, REV>(p, behind, stream); st != LA_OK) return st;
    return launch_behind(true, la::gated_prefix_kernel, dim3((unsigned)(pl.tab.S * p.H), D * D / 1024), 256, 0, stream,
                         reinterpret_cast<float4 *>(p.seg_out), p.seg_total,
                         reinterpret_cast<const float4 *>(initial), nullptr, p.H, D * D / 4, REV ? 1 : 0, pl.tab);
}

template <int D, bool REV>
la_status gated_states_tc(const void *a, const void *b, const void *g, const float *initial, void *snap,
                          const void *other, float *through, float *fin, int H, long long T, const GatedPlan &pl,
                          uint8_t *ws, bool behind, cudaStream_t stream) {
    la::GatedStateParams p;
    const long long rows = 2ll * pl.tab.blocks * H * D;  // two parts
    if (!fill_gated_states<D>(p, a, b, g, H, T, pl) ||
        (snap != nullptr && !make_map(&p.tmap_snap, snap, rows, 1, D, D)) ||
        (through != nullptr && !make_map(&p.tmap_other, other, rows, 1, D, D)))
        return LA_ERR_CUDA;
    if (pl.segmented) {
        float *seg_in = nullptr;
        if (la_status st = gated_seg_states_tc<D, REV>(p, initial, pl, ws, behind, stream, seg_in); st != LA_OK) return st;
        p.seg_in = seg_in;
    }
    p.initial = initial;
    p.fin = fin;
    p.have_snap = snap != nullptr;
    p.through = through;
    return launch_gated_states<D, REV>(p, behind || pl.segmented, stream);
}

// Final states of sequences without tokens: their initial states.
la_status gated_no_tokens(const float *initial, float *fin, int S, int H, int D, cudaStream_t stream) {
    if (fin == nullptr || fin == initial) return LA_OK;
    if (initial == nullptr)
        la::state_zero_kernel<<<(unsigned)(S * H), 256, 0, stream>>>(reinterpret_cast<float4 *>(fin), D * D / 4);
    else
        la::state_copy_kernel<<<(unsigned)(S * H), 256, 0, stream>>>(reinterpret_cast<const float4 *>(initial),
                                                                     reinterpret_cast<float4 *>(fin), nullptr, H,
                                                                     D * D / 4, S);
    return launched();
}

template <int D>
la_status gated_prefill_tc(const void *q, const void *k, const void *v, const void *g, void *o, const float *state_in,
                           float *state_out, int H, long long T, const GatedPlan &pl, uint8_t *ws,
                           cudaStream_t stream) {
    using C = la::GatedPrefillCfg<D>;
    auto kern = la::gated_prefill_tc_kernel<D>;
    static std::atomic<bool> fits{false};
    if (!starts_with(kern, C::R_LAUNCH, fits)) return LA_ERR_CUDA;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess)
        return LA_ERR_CUDA;
    la::GatedPrefillParams p;
    std::memset(&p, 0, sizeof p);
    if (!make_map(&p.tmap_q, q, T, H, D, C::C) || !make_map(&p.tmap_k, k, T, H, D, C::C) ||
        !make_map(&p.tmap_v, v, T, H, D, C::C) || !make_map(&p.tmap_o, o, T, H, D, 32))
        return LA_ERR_CUDA;
    if (pl.segmented) {
        la::GatedStateParams sp;
        float *seg_in = nullptr;
        if (!fill_gated_states<D>(sp, k, v, g, H, T, pl)) return LA_ERR_CUDA;
        if (la_status st = gated_seg_states_tc<D, false>(sp, state_in, pl, ws, false, stream, seg_in); st != LA_OK)
            return st;
        p.seg_in = seg_in;
    }
    p.g = static_cast<const __nv_bfloat16 *>(g);
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.initial = state_in;
    p.fin = state_out;
    p.H = H;
    p.timeout_ns = kWaitLimitNs;
    p.tab = pl.tab;
    // Started early, the two slices of a head land on SMs as these come free, not side by side,
    // which slows a long pass more than it saves.  8 heads, D = 128, with and without: 15 blocks a
    // segment 75 and 78 us, 29 123 and 125, 43 171 and 173; 57 240 and 225, 86 383 and 365, 114 492
    // and 486.  (4 heads: 29 blocks 147 and 153, 57 257 and 257; D = 64: within the noise.)
    const bool behind = pl.segmented && pl.tab.seg_blocks <= 48;
    return launch_behind(behind, kern, dim3((unsigned)(pl.tab.segs * H * C::NVS)), C::THREADS, C::SMEM_BYTES,
                         stream, p);
}

template <int D>
la_status gated_backward_tc(const void *q, const void *k, const void *v, const void *g, const void *dout, void *dq,
                            void *dk, void *dv, void *dg, const float *state_in, const float *d_state,
                            float *d_state_in, int H, long long T, const GatedPlan &pl, uint8_t *ws,
                            cudaStream_t stream) {
    using C = la::GatedBackwardCfg<D>;
    using bf = __nv_bfloat16;
    void *snap = nullptr, *dsnap = nullptr;
    float *through = nullptr;
    if (pl.longest > 1 || state_in != nullptr) snap = ws + pl.snap;
    if (pl.longest > 1 || d_state != nullptr) dsnap = ws + pl.dsnap;
    if (snap != nullptr && dsnap != nullptr && dg != nullptr) through = reinterpret_cast<float *>(ws + pl.through);
    if (snap != nullptr)
        if (la_status st = gated_states_tc<D, false>(k, v, g, state_in, snap, nullptr, nullptr, nullptr, H, T, pl, ws,
                                                     false, stream);
            st != LA_OK)
            return st;
    if (dsnap != nullptr || d_state_in != nullptr)
        if (la_status st = gated_states_tc<D, true>(q, dout, g, d_state, dsnap, snap, through, d_state_in, H, T, pl,
                                                    ws, snap != nullptr, stream);
            st != LA_OK)
            return st;
    la::GatedBackwardParams p;
    std::memset(&p, 0, sizeof p);
    const long long rows = 2ll * pl.tab.blocks * H * D;  // two parts
    if (!make_map(&p.tmap_q, q, T, H, D, C::C) || !make_map(&p.tmap_k, k, T, H, D, C::C) ||
        !make_map(&p.tmap_v, v, T, H, D, C::C) || !make_map(&p.tmap_do, dout, T, H, D, C::C) ||
        (snap != nullptr && !make_map(&p.tmap_s, snap, rows, 1, D, D)) ||
        (dsnap != nullptr && !make_map(&p.tmap_ds, dsnap, rows, 1, D, D)))
        return LA_ERR_CUDA;
    p.g = static_cast<const bf *>(g);
    p.through = through;
    p.dq = static_cast<bf *>(dq);
    p.dk = static_cast<bf *>(dk);
    p.dv = static_cast<bf *>(dv);
    p.dg = static_cast<bf *>(dg);
    p.H = H;
    p.have_s = snap != nullptr;
    p.have_ds = dsnap != nullptr;
    p.timeout_ns = kWaitLimitNs;
    p.tab = pl.tab;
    auto kern = la::gated_backward_tc_kernel<D>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess)
        return LA_ERR_CUDA;
    return launch_behind(snap != nullptr || dsnap != nullptr || d_state_in != nullptr, kern,
                         dim3((unsigned)std::min(kSMs, pl.tab.blocks * H)), C::THREADS, C::SMEM_BYTES, stream, p);
}

// Checks that the gated sequence operators share.
la_status check_gated(int B, int H, int N, int D, unsigned flags) {
    if (flags & ~(unsigned)LA_BF16) return LA_ERR_INVALID_ARG;
    if (H < 1 || N < 0 || B < 1) return LA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

bool aligned_gate(const void *p, unsigned flags) {
    return (reinterpret_cast<uintptr_t>(p) & ((flags & LA_BF16) ? 1u : 3u)) == 0;
}

}  // namespace

extern "C" {

const char *la_status_string(la_status s) {
    switch (s) {
        case LA_OK: return "LA_OK";
        case LA_ERR_INVALID_ARG: return "LA_ERR_INVALID_ARG";
        case LA_ERR_UNSUPPORTED: return "LA_ERR_UNSUPPORTED";
        case LA_ERR_CUDA: return "LA_ERR_CUDA";
        case LA_ERR_DEVICE_TIMEOUT: return "LA_ERR_DEVICE_TIMEOUT";
        case LA_ERR_DEVICE_RANGE: return "LA_ERR_DEVICE_RANGE";
    }
    return "LA_ERR_UNKNOWN";
}

int la_version(void) { return 200; }

la_status la_prefill(const void *q, const void *k, const void *v, void *o, int B, int H, int N,
                     int D, int beta, const int32_t *cu_seqlens, int num_seqs, unsigned flags,
                     float *state_ws, void *stream_) {
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    const unsigned known = LA_BF16 | LA_OUT_RMSNORM | LA_WRITE_STATE | LA_READ_STATE;
    if (flags & ~known) return LA_ERR_INVALID_ARG;
    if (H < 1 || N < 0 || B < 1) return LA_ERR_INVALID_ARG;
    // with no tokens (N == 0) the data pointers are never used and may be NULL
    if (N > 0 && (!q || !k || !v || !o)) return LA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return LA_ERR_INVALID_ARG;
    const bool want_state = (flags & LA_WRITE_STATE) != 0;
    const bool read_state = (flags & LA_READ_STATE) != 0;
    if ((want_state || read_state) && (state_ws == nullptr || !aligned16(state_ws)))
        return LA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return LA_ERR_UNSUPPORTED;
    if (beta != 64 && beta != 128) return LA_ERR_UNSUPPORTED;

    // Sequence table (host-validated).
    SeqTable seqs;
    long long T = 0;
    int S = 0;
    if (la_status st = build_seq_table(B, N, cu_seqlens, num_seqs, seqs, T, S); st != LA_OK)
        return st;
    if (T >= (1ll << 31) || (long long)S * H * 2 >= (1ll << 31)) return LA_ERR_UNSUPPORTED;
    if (S == 0 || H == 0) return LA_OK;

    const int rms = (flags & LA_OUT_RMSNORM) ? 1 : 0;
    float *state = want_state ? state_ws : nullptr;
    const float *state_in = read_state ? state_ws : nullptr;
    if (T == 0) {
        // Every sequence is empty: its final state is its initial state, already in
        // place with LA_READ_STATE, else zero.
        if (want_state && !read_state) {
            la::state_zero_kernel<<<(unsigned)(S * H), 256, 0, stream>>>(
                reinterpret_cast<float4 *>(state_ws), D * D / 4);
            return cudaGetLastError() == cudaSuccess ? LA_OK : LA_ERR_CUDA;
        }
        return LA_OK;
    }

    if (flags & LA_BF16) {
        // Sequences of one token are decode steps: they go to the decode kernel (reading
        // their rows of the packed arrays in place), the rest to the prefill kernel.  A
        // one-token sequence would otherwise hold a whole prefill CTA (pair) for one row.
        la::OneTokenTable ot;
        ot.identity = 0;
        int n1 = 0;
        if (seqs.varlen) {
            int w = 0;
            for (int r = 0; r < S; ++r) {
                if (seqs.seq_len[r] == 1) {
                    ot.row[n1] = seqs.seq_start[r];
                    ot.sid[n1] = seqs.seq_id[r];
                    ++n1;
                } else {
                    seqs.seq_start[w] = seqs.seq_start[r];
                    seqs.seq_len[w] = seqs.seq_len[r];
                    seqs.seq_id[w] = seqs.seq_id[r];
                    ++w;
                }
            }
            S = w;
        } else if (N == 1) {
            ot.identity = 1;
            n1 = S;
            S = 0;
        }
        if (n1 > 0) {
            using bf = __nv_bfloat16;
            const bf *qb = static_cast<const bf *>(q), *kb = static_cast<const bf *>(k),
                     *vb = static_cast<const bf *>(v);
            bf *ob = static_cast<bf *>(o);
            float *ws = (want_state || read_state) ? state_ws : nullptr;
            if (D == 128)
                la::decode_rows_kernel<128, bf><<<(unsigned)(n1 * H), 256, 0, stream>>>(
                    qb, kb, vb, ob, ws, H, read_state ? 1 : 0, want_state ? 1 : 0, rms, ot);
            else
                la::decode_rows_kernel<64, bf><<<(unsigned)(n1 * H), 256, 0, stream>>>(
                    qb, kb, vb, ob, ws, H, read_state ? 1 : 0, want_state ? 1 : 0, rms, ot);
            if (cudaGetLastError() != cudaSuccess) return LA_ERR_CUDA;
        }
        if (S == 0) return LA_OK;
        const long long Tm = T;
        if (beta == 128 && D == 128) {
            // paired-CTA kernel: each CTA of a pair loads half of the rows / columns
            la::PrefillPairParams pp;
            std::memset(&pp, 0, sizeof pp);
            if (!make_map(&pp.tmap_q64, q, Tm, H, D, 64) || !make_map(&pp.tmap_k64, k, Tm, H, D, 64) ||
                !make_map(&pp.tmap_k128, k, Tm, H, D, 128) || !make_map(&pp.tmap_v128, v, Tm, H, D, 128) ||
                !make_map(&pp.tmap_o32, o, Tm, H, D, 32))
                return LA_ERR_CUDA;
            pp.o = static_cast<__nv_bfloat16 *>(o);
            pp.state = state;
            pp.state_in = state_in;
            pp.H = H;
            pp.rmsnorm = rms;
            pp.timeout_ns = kWaitLimitNs;
            pp.seqs = seqs;
            return launch_pair(pp, S * H, stream);
        }
        PrefillTcParams p;
        std::memset(&p, 0, sizeof p);
        if (!make_map(&p.tmap_q, q, Tm, H, D, beta) || !make_map(&p.tmap_k, k, Tm, H, D, beta) ||
            !make_map(&p.tmap_v, v, Tm, H, D, beta))
            return LA_ERR_CUDA;
        p.o = static_cast<__nv_bfloat16 *>(o);
        p.state = state;
        p.state_in = state_in;
        p.H = H;
        p.rmsnorm = rms;
        p.timeout_ns = kWaitLimitNs;
        p.seqs = seqs;
        const int units = S * H * (D / 64);
        if (beta == 64 && D == 128) return launch_tc<64, 128>(p, units, stream);
        if (beta == 128 && D == 64) return launch_tc<128, 64>(p, units, stream);
        return launch_tc<64, 64>(p, units, stream);
    }
    const float *qf = static_cast<const float *>(q), *kf = static_cast<const float *>(k),
                *vf = static_cast<const float *>(v);
    float *of = static_cast<float *>(o);
    if (beta == 128 && D == 128) return launch_simt<128, 128>(qf, kf, vf, of, state, state_in, H, rms, seqs, S, stream);
    if (beta == 64 && D == 128) return launch_simt<64, 128>(qf, kf, vf, of, state, state_in, H, rms, seqs, S, stream);
    if (beta == 128 && D == 64) return launch_simt<128, 64>(qf, kf, vf, of, state, state_in, H, rms, seqs, S, stream);
    return launch_simt<64, 64>(qf, kf, vf, of, state, state_in, H, rms, seqs, S, stream);
}

la_status la_chunk_state(const void *k, const void *v, int B, int H, int N, int D,
                         const int32_t *cu_seqlens, int num_seqs, unsigned flags, float *state_out,
                         void *stream_) {
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (flags & ~(unsigned)LA_BF16) return LA_ERR_INVALID_ARG;
    if (H < 1 || N < 0 || B < 1) return LA_ERR_INVALID_ARG;
    if (N > 0 && (!k || !v)) return LA_ERR_INVALID_ARG;
    if (!state_out) return LA_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(state_out)) return LA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return LA_ERR_UNSUPPORTED;
    SeqTable seqs;
    long long T = 0;
    int S = 0;
    if (la_status st = build_seq_table(B, N, cu_seqlens, num_seqs, seqs, T, S); st != LA_OK)
        return st;
    if (T >= (1ll << 31) || (long long)S * H * 2 >= (1ll << 31)) return LA_ERR_UNSUPPORTED;
    if (S == 0) return LA_OK;
    if (T == 0) {  // every sequence is empty: zero states
        la::state_zero_kernel<<<(unsigned)(S * H), 256, 0, stream>>>(
            reinterpret_cast<float4 *>(state_out), D * D / 4);
        return cudaGetLastError() == cudaSuccess ? LA_OK : LA_ERR_CUDA;
    }
    if (flags & LA_BF16) {
        la::ChunkStateParams p;
        std::memset(&p, 0, sizeof p);
        if (!make_map(&p.tmap_k, k, T, H, D, 128) || !make_map(&p.tmap_v, v, T, H, D, 128))
            return LA_ERR_CUDA;
        p.state = state_out;
        p.H = H;
        p.timeout_ns = kWaitLimitNs;
        p.seqs = seqs;
        auto launch = [&](auto kern, int smem, int threads, int nvs) -> la_status {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
                cudaSuccess)
                return LA_ERR_CUDA;
            kern<<<(unsigned)(S * H * nvs), threads, smem, stream>>>(p);
            return cudaGetLastError() == cudaSuccess ? LA_OK : LA_ERR_CUDA;
        };
        if (D == 128)
            return launch(la::chunk_state_tc_kernel<128>, la::ChunkCfg<128>::SMEM_BYTES,
                          la::ChunkCfg<128>::THREADS, la::ChunkCfg<128>::NVS);
        return launch(la::chunk_state_tc_kernel<64>, la::ChunkCfg<64>::SMEM_BYTES,
                      la::ChunkCfg<64>::THREADS, la::ChunkCfg<64>::NVS);
    }
    const float *kf = static_cast<const float *>(k), *vf = static_cast<const float *>(v);
    auto launch_simt_state = [&](auto kern, int Dv) -> la_status {
        const int smem = (2 * 64 * Dv + Dv * Dv) * 4;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return LA_ERR_CUDA;
        kern<<<(unsigned)(S * H), 256, smem, stream>>>(kf, vf, state_out, H, seqs);
        return cudaGetLastError() == cudaSuccess ? LA_OK : LA_ERR_CUDA;
    };
    if (D == 128) return launch_simt_state(la::chunk_state_simt_kernel<128>, 128);
    return launch_simt_state(la::chunk_state_simt_kernel<64>, 64);
}

la_status la_state_prefix(const float *gathered, int R, int rank, int S, int H, int D, float *out,
                          void *stream_) {
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (R < 1 || rank < 0 || rank > R || S < 0 || H < 1) return LA_ERR_INVALID_ARG;
    if (!gathered || !out || !aligned16(gathered) || !aligned16(out)) return LA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return LA_ERR_UNSUPPORTED;
    if ((long long)S * H >= (1ll << 31)) return LA_ERR_UNSUPPORTED;
    if (S == 0) return LA_OK;
    const int n4 = D * D / 4;
    la::state_prefix_kernel<<<(unsigned)(S * H), 256, 0, stream>>>(
        reinterpret_cast<const float4 *>(gathered), reinterpret_cast<float4 *>(out), rank,
        (size_t)S * H * n4, n4);
    return cudaGetLastError() == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

la_status la_selftest_wait(unsigned long long limit_ns, void *stream_) {
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (limit_ns < 1000ull) limit_ns = 1000ull;
    if (limit_ns > kWaitLimitNs) limit_ns = kWaitLimitNs;
    la::selftest_wait_kernel<<<1, 32, 0, stream>>>(limit_ns);
    return cudaGetLastError() == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

la_status la_decode_step(const void *q, const void *k, const void *v, float *state, void *o, int B,
                         int H, int D, unsigned flags, void *stream_) {
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    const unsigned known = LA_BF16 | LA_OUT_RMSNORM;
    if (flags & ~known) return LA_ERR_INVALID_ARG;
    if (B < 0 || H < 1) return LA_ERR_INVALID_ARG;
    if (!q || !k || !v || !o || !state) return LA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(state))
        return LA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return LA_ERR_UNSUPPORTED;
    if ((long long)B * H >= (1ll << 31)) return LA_ERR_UNSUPPORTED;
    if (B == 0) return LA_OK;
    const int rms = (flags & LA_OUT_RMSNORM) ? 1 : 0;
    const unsigned grid = (unsigned)(B * H);
    if (flags & LA_BF16) {
        using T = __nv_bfloat16;
        if (D == 128)
            la::decode_step_kernel<128, T><<<grid, 256, 0, stream>>>(
                (const T *)q, (const T *)k, (const T *)v, state, (T *)o, rms);
        else
            la::decode_step_kernel<64, T><<<grid, 256, 0, stream>>>(
                (const T *)q, (const T *)k, (const T *)v, state, (T *)o, rms);
    } else {
        if (D == 128)
            la::decode_step_kernel<128, float><<<grid, 256, 0, stream>>>(
                (const float *)q, (const float *)k, (const float *)v, state, (float *)o, rms);
        else
            la::decode_step_kernel<64, float><<<grid, 256, 0, stream>>>(
                (const float *)q, (const float *)k, (const float *)v, state, (float *)o, rms);
    }
    return cudaGetLastError() == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

la_status la_state_out(const float *state_ws, float *state_dst, int S, int H, int D,
                       const int32_t *seq_to_slot, int num_slots, void *stream_) {
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (S < 0 || H < 1 || num_slots < 0) return LA_ERR_INVALID_ARG;
    if (!state_ws || !state_dst) return LA_ERR_INVALID_ARG;
    if (!aligned16(state_ws) || !aligned16(state_dst)) return LA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return LA_ERR_UNSUPPORTED;
    if (seq_to_slot == nullptr && S > num_slots) return LA_ERR_INVALID_ARG;
    if ((long long)S * H >= (1ll << 31)) return LA_ERR_UNSUPPORTED;
    if (S == 0) return LA_OK;
    la::state_copy_kernel<<<(unsigned)(S * H), 256, 0, stream>>>(
        reinterpret_cast<const float4 *>(state_ws), reinterpret_cast<float4 *>(state_dst),
        seq_to_slot, H, D * D / 4, num_slots);
    return cudaGetLastError() == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

la_status la_gated_workspace(int B, int H, int N, int D, const int32_t *cu_seqlens, int num_seqs, unsigned flags,
                             int backward, unsigned long long *bytes) {
    if (bytes == nullptr) return LA_ERR_INVALID_ARG;
    if (la_status st = check_gated(B, H, N, D, flags); st != LA_OK) return st;
    GatedPlan pl;
    long long T = 0;
    if (la_status st = plan_gated(B, H, N, D, cu_seqlens, num_seqs, flags, backward != 0, pl, T); st != LA_OK)
        return st;
    *bytes = pl.bytes;
    return LA_OK;
}

la_status la_gated_prefill(const void *q, const void *k, const void *v, const void *g, void *o, int B, int H, int N,
                           int D, const int32_t *cu_seqlens, int num_seqs, unsigned flags, const float *state_in,
                           float *state_out, void *workspace, unsigned long long workspace_bytes, void *stream_) {
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (la_status st = check_gated(B, H, N, D, flags); st != LA_OK) return st;
    if (N > 0 && (!q || !k || !v || !o)) return LA_ERR_INVALID_ARG;
    for (const void *p : {q, k, v, (const void *)o, (const void *)state_in, (const void *)state_out,
                          (const void *)workspace})
        if (!aligned16(p)) return LA_ERR_INVALID_ARG;
    if (!aligned_gate(g, flags)) return LA_ERR_INVALID_ARG;
    GatedPlan pl;
    long long T = 0;
    if (la_status st = plan_gated(B, H, N, D, cu_seqlens, num_seqs, flags, false, pl, T); st != LA_OK) return st;
    if (pl.bytes > workspace_bytes || (pl.bytes > 0 && workspace == nullptr)) return LA_ERR_INVALID_ARG;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (T == 0) return gated_no_tokens(state_in, state_out, pl.tab.S, H, D, stream);
    if (pl.ones > 0) {
        auto *rows = (flags & LA_BF16) ? (D == 128 ? gated_rows<128, __nv_bfloat16> : gated_rows<64, __nv_bfloat16>)
                                       : (D == 128 ? gated_rows<128, float> : gated_rows<64, float>);
        if (la_status st = rows(q, k, v, g, o, state_in, state_out, H, pl, stream); st != LA_OK || pl.tab.S == 0)
            return st;
    }
    if (flags & LA_BF16) {
        if (D == 128) return gated_prefill_tc<128>(q, k, v, g, o, state_in, state_out, H, T, pl, ws, stream);
        return gated_prefill_tc<64>(q, k, v, g, o, state_in, state_out, H, T, pl, ws, stream);
    }
    const float *qf = static_cast<const float *>(q), *kf = static_cast<const float *>(k),
                *vf = static_cast<const float *>(v), *gf = static_cast<const float *>(g);
    float *of = static_cast<float *>(o);
    if (D == 128) return gated_prefill_simt<128>(qf, kf, vf, gf, of, state_in, state_out, H, pl, ws, stream);
    return gated_prefill_simt<64>(qf, kf, vf, gf, of, state_in, state_out, H, pl, ws, stream);
}

la_status la_gated_prefill_backward(const void *q, const void *k, const void *v, const void *g, const void *dout,
                                    void *dq, void *dk, void *dv, void *dg, int B, int H, int N, int D,
                                    const int32_t *cu_seqlens, int num_seqs, unsigned flags, const float *state_in,
                                    const float *d_state, float *d_state_in, void *workspace,
                                    unsigned long long workspace_bytes, void *stream_) {
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (la_status st = check_gated(B, H, N, D, flags); st != LA_OK) return st;
    if (N > 0 && (!q || !k || !v || !dout || !dq || !dk || !dv)) return LA_ERR_INVALID_ARG;
    if (dg != nullptr && g == nullptr) return LA_ERR_INVALID_ARG;
    for (const void *p : {q, k, v, dout, (const void *)dq, (const void *)dk, (const void *)dv,
                          (const void *)state_in, (const void *)d_state, (const void *)d_state_in,
                          (const void *)workspace})
        if (!aligned16(p)) return LA_ERR_INVALID_ARG;
    if (!aligned_gate(g, flags) || !aligned_gate(dg, flags)) return LA_ERR_INVALID_ARG;
    GatedPlan pl;
    long long T = 0;
    if (la_status st = plan_gated(B, H, N, D, cu_seqlens, num_seqs, flags, true, pl, T); st != LA_OK) return st;
    if (pl.bytes > workspace_bytes || (pl.bytes > 0 && workspace == nullptr)) return LA_ERR_INVALID_ARG;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (T == 0) return gated_no_tokens(d_state, d_state_in, pl.tab.S, H, D, stream);
    auto *run = pl.simt ? ((flags & LA_BF16) ? (D == 128 ? gated_backward_simt<128, __nv_bfloat16>
                                                         : gated_backward_simt<64, __nv_bfloat16>)
                                             : (D == 128 ? gated_backward_simt<128, float>
                                                         : gated_backward_simt<64, float>))
                        : nullptr;
    if (run != nullptr)
        return run(q, k, v, g, dout, dq, dk, dv, dg, state_in, d_state, d_state_in, H, pl, ws, stream);
    if (D == 128)
        return gated_backward_tc<128>(q, k, v, g, dout, dq, dk, dv, dg, state_in, d_state, d_state_in, H, T, pl, ws,
                                      stream);
    return gated_backward_tc<64>(q, k, v, g, dout, dq, dk, dv, dg, state_in, d_state, d_state_in, H, T, pl, ws, stream);
}

la_status la_gated_decode_step(const void *q, const void *k, const void *v, const void *g, float *state, void *o,
                               int B, int H, int D, const int32_t *slots, int num_slots, unsigned flags,
                               void *stream_) {
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (flags & ~(unsigned)LA_BF16) return LA_ERR_INVALID_ARG;
    if (B < 0 || H < 1 || num_slots < 0) return LA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return LA_ERR_UNSUPPORTED;
    if (B == 0) return LA_OK;
    if (!q || !k || !v || !o || !state) return LA_ERR_INVALID_ARG;
    for (const void *p : {q, k, v, (const void *)o, (const void *)state})
        if (!aligned16(p)) return LA_ERR_INVALID_ARG;
    if (!aligned_gate(g, flags) || (reinterpret_cast<uintptr_t>(slots) & 3u)) return LA_ERR_INVALID_ARG;
    if (slots == nullptr && num_slots < B) return LA_ERR_INVALID_ARG;
    if (slots != nullptr && B > LA_MAX_SLOT_ROWS) return LA_ERR_UNSUPPORTED;
    if ((long long)B * H >= (1ll << 31)) return LA_ERR_UNSUPPORTED;
    const unsigned grid = (unsigned)(B * H);
    auto run = [&](auto *x) {
        using E = std::remove_pointer_t<decltype(x)>;
        const E *qe = static_cast<const E *>(q), *ke = static_cast<const E *>(k), *ve = static_cast<const E *>(v),
                *ge = static_cast<const E *>(g);
        E *oe = static_cast<E *>(o);
        if (D == 128)
            la::gated_decode_kernel<128, E><<<grid, 256, 0, stream>>>(qe, ke, ve, ge, state, oe, H, slots, num_slots);
        else
            la::gated_decode_kernel<64, E><<<grid, 256, 0, stream>>>(qe, ke, ve, ge, state, oe, H, slots, num_slots);
        return launched();
    };
    if (flags & LA_BF16) return run(static_cast<__nv_bfloat16 *>(nullptr));
    return run(static_cast<float *>(nullptr));
}

la_status la_get_device_status(void *stream_) {
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (cudaStreamSynchronize(stream) != cudaSuccess) return LA_ERR_CUDA;
    unsigned int word = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&word, la::g_device_status, sizeof word) != cudaSuccess)
        return LA_ERR_CUDA;
    if (word != 0 && cudaMemcpyToSymbol(la::g_device_status, &zero, sizeof zero) != cudaSuccess)
        return LA_ERR_CUDA;
    if (word == la::DEV_TIMEOUT) return LA_ERR_DEVICE_TIMEOUT;
    if (word == la::DEV_RANGE) return LA_ERR_DEVICE_RANGE;
    return LA_OK;
}

}  // extern "C"
