// Gated lightning attention: the tables, the small kernels and the fp32 kernels.
//
// With a log-decay g_t per token and head the recurrence and its readout are
//     S_t = e^{g_t} S_{t-1} + k_t v_t^T,     o_t = S_t^T q_t.
// A sequence is cut into blocks of C tokens.  With G_i the sum of g over the block's
// tokens up to and including i, and S the state at the block's start,
//     o_i = sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j  +  e^{G_i} S^T q_i,
//     S  <- e^{G_C} S + sum_j e^{G_C - G_j} k_j v_j^T.
// Only differences of G enter, and never as a quotient of two exponentials: with g <= 0
// every factor is at most 1, however fast the state decays.
//
// Backward, with dS the gradient of the state at the block's end (from the end of the
// sequence towards its start dS <- e^{G_C} dS + sum_i e^{G_i} q_i do_i^T):
//     P_ij = e^{G_i - G_j} (q_i . k_j),  dP_ij = e^{G_i - G_j} (do_i . v_j)     (j <= i)
//     dq = dP k    + e^{G_i} S do_i
//     dk = dP^T q  + e^{G_C - G_j} dS v_j
//     dv = P^T do  + e^{G_C - G_j} dS^T k_j
//     dg_t = sum over the pairs (j < t <= i), j and i anywhere, of the pair's share of the
//            loss, W_ij = dP_ij (q_i . k_j):
//            both in the block:            sum_{j < t <= i} W_ij
//            j before the block:           sum_{i >= t} q_i . (e^{G_i} S do_i)
//            i behind the block:           sum_{j < t} k_j . (e^{G_C - G_j} dS v_j)
//            both outside:                 e^{G_C} <dS, S>
//            Every term is a sum over pairs that span t.  (The running sum of
//            q.dq - k.dk over a whole sequence is the same number, left over when the
//            shares of all pairs that do not span t cancel: rounding grows with the
//            length of the sequence there, here it does not.)
#pragma once

#include "decode.cuh"
#include "prefill_tc.cuh"

namespace la {

// The sequences of a call (longest first) with their blocks and segments.  Blocks of C
// tokens are numbered through the call; a segment is seg_blocks consecutive blocks of one
// sequence (every sequence has at least one, an empty one of no blocks).
struct GatedTable {
    SeqTable seqs;
    int S;
    int C;               // tokens per block
    int seg_blocks;
    int blocks, segs;    // totals
    int blocks_per_seq, segs_per_seq;        // uniform batches
    int block0[LA_MAX_VARLEN_SEQS + 1];      // packed batches: prefix sums by rank
    int seg0[LA_MAX_VARLEN_SEQS + 1];

    // Rank of the sequence that entry x of the prefix array lies in.
    __device__ __forceinline__ int find(const int *prefix, int x) const {
        int lo = 0, hi = S;  // prefix[lo] <= x < prefix[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid] <= x)
                lo = mid;
            else
                hi = mid;
        }
        return lo;
    }
    // Block x: its sequence's rank and its number in the sequence.
    __device__ __forceinline__ void block(int x, int &rank, int &b) const {
        if (seqs.varlen) {
            rank = find(block0, x);
            b = x - block0[rank];
        } else {
            rank = x / blocks_per_seq;
            b = x - rank * blocks_per_seq;
        }
    }
    __device__ __forceinline__ void seg(int x, int &rank, int &s) const {
        if (seqs.varlen) {
            rank = find(seg0, x);
            s = x - seg0[rank];
        } else {
            rank = x / segs_per_seq;
            s = x - rank * segs_per_seq;
        }
    }
    __device__ __forceinline__ int first_block(int rank) const {
        return seqs.varlen ? block0[rank] : rank * blocks_per_seq;
    }
    __device__ __forceinline__ int first_seg(int rank) const {
        return seqs.varlen ? seg0[rank] : rank * segs_per_seq;
    }
    __device__ __forceinline__ int num_segs(int rank) const {
        return seqs.varlen ? seg0[rank + 1] - seg0[rank] : segs_per_seq;
    }
};

// A log-decay as the kernels use it.  e^{-110} is 0 in fp32, as e^{-inf} is; a finite bound
// keeps differences of sums defined, and a small one keeps them exact: 128 such tokens sum to
// 2^14, whose rounding is 2^-10.  A NaN stays one.
__device__ __forceinline__ float clamp_gate(float g) { return g < -110.f ? -110.f : g; }

// The kernels of one call overlap at their ends: each lets the next one's CTAs start as SMs
// come free (next_may_start) and set up their shared memory and TMEM, which then wait for
// all that the kernel before has written (previous_done) before they touch global memory.
// What an earlier kernel of the call writes is no `const __restrict__` argument of a later
// one: it changes while that one's CTAs already exist, and must not be read as constant.
// (Replayed from a graph, a backward call of 4096 tokens, 16 heads, D = 64: 72 us instead of 74;
// of 128 tokens, 64 heads, D = 128, with states 29 instead of 30.)
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void previous_done() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// out = start states of a (sequence, head)'s segments from their own end states, in order:
//     X_0 = initial, X_{s+1} = e^{total_s} X_s + local_s;   seg_state[s] <- X_s.
// `rev` walks the segments from the last to the first (the state's gradient).  One thread
// per float4 of the state; grid (S * H, D * D / 1024).  Latency-bound: eight segments' loads
// are in flight at once.  `fin` (or nullptr) takes the state behind the last one; it may be
// `initial`.
__global__ void __launch_bounds__(256)
    gated_prefix_kernel(float4 *seg_state, const float *seg_total,
                        const float4 *initial, float4 *fin, int H, int n4, int rev,
                        const __grid_constant__ GatedTable tab) {
    const int rank = blockIdx.x / H, h = blockIdx.x % H;
    const int x = blockIdx.y * 256 + threadIdx.x;
    next_may_start();
    previous_done();
    int start, len, sid;
    tab.seqs.get(rank, start, len, sid);
    const int s0 = tab.first_seg(rank), ns = tab.num_segs(rank);
    float4 X = initial != nullptr ? initial[((size_t)sid * H + h) * n4 + x] : make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int N = 8;  // segments in flight: their loads do not wait for one another
    for (int t0 = 0; t0 < ns; t0 += N) {
        float4 l[N];
        float a[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int t = t0 + e;
            const size_t at = (size_t)(s0 + (rev ? ns - 1 - t : t)) * H + h;
            if (t < ns) l[e] = seg_state[at * n4 + x], a[e] = seg_total[at];
        }
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int t = t0 + e;
            if (t >= ns) break;
            const float w = expf(a[e]);
            seg_state[((size_t)(s0 + (rev ? ns - 1 - t : t)) * H + h) * n4 + x] = X;
            X = make_float4(fmaf(w, X.x, l[e].x), fmaf(w, X.y, l[e].y), fmaf(w, X.z, l[e].z), fmaf(w, X.w, l[e].w));
        }
    }
    if (fin != nullptr) fin[((size_t)sid * H + h) * n4 + x] = X;
}

// ------------------------------------------------------------------ CUDA-core kernels (fp32)
// Blocks of 64 tokens, 256 threads, tiles staged in shared memory.
struct GatedSimt {
    static constexpr int C = 64;
    static constexpr int THREADS = 256;
    static constexpr int VS = 32;  // state columns per CTA of the state kernel
};

// Sums of the block's log-decays: sG[i] = g_0 + .. + g_i (i < nv; rows behind the sequence
// repeat the last sum), in fp64, so that differences of two large sums stay exact to fp32.
// Called by one warp.
template <typename E>
__device__ __forceinline__ void simt_gate_sums(double *sG, const E *__restrict__ g, int row0, int nv,
                                               int H, int h) {
    const int lane = threadIdx.x & 31;
    double carry = 0.0;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int i = 32 * half + lane;
        double x = i < nv && g != nullptr ? (double)clamp_gate(to_f32(g[(size_t)(row0 + i) * H + h])) : 0.0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        x += carry;
        sG[i] = x;
        carry = __shfl_sync(0xffffffffu, x, 31);
    }
}

__device__ __forceinline__ void cp_async16(float *dst, const float *src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(real ? 16 : 0)
                 : "memory");
}
// Four elements to shared memory as fp32, zeros where `real` is not: fp32 by cp.async, bf16
// through registers.
__device__ __forceinline__ void simt_load4(float *dst, const float *src, bool real) { cp_async16(dst, src, real); }
__device__ __forceinline__ void simt_load4(float *dst, const __nv_bfloat16 *src, bool real) {
    const uint2 v = real ? *reinterpret_cast<const uint2 *>(src) : make_uint2(0u, 0u);
    *reinterpret_cast<float4 *>(dst) = make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                                                   __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
}
__device__ __forceinline__ void simt_store4(float *dst, float a, float b, float c, float d) {
    *reinterpret_cast<float4 *>(dst) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void simt_store4(__nv_bfloat16 *dst, float a, float b, float c, float d) {
    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The state scan: one CTA per (segment, head, VS state columns).
//   forward (REV = false): X = state,           X <- e^{G_C} X + sum_j e^{G_C - G_j} k_j v_j^T
//   reverse (REV = true):  X = state gradient,  X <- e^{G_C} X + sum_i e^{G_i} q_i do_i^T
// (a, b) = (k, v) or (q, do).  The state before each update goes to snap[block][h]; a
// segment starts from seg_in (segmented call) or the sequence's initial state; seg_out and
// seg_total take a segment's own end state and decay; fin the sequence's final state.
// The next block's tiles come by cp.async while this one is added up: a block of few heads is
// all latency (64 x 64 x 32 products a CTA; about 3 us a block).
template <int D>
struct GatedStateSimt {
    static constexpr int A = GatedSimt::C * D, B = GatedSimt::C * GatedSimt::VS;
    static constexpr int SMEM_BYTES = 2 * (A + B) * 4;
    static constexpr int THREADS = GatedSimt::THREADS + 32;  // one warp forms the gate sums
};

template <int D, bool REV, typename E>
__global__ void __launch_bounds__(GatedStateSimt<D>::THREADS)
    gated_state_simt_kernel(const E *__restrict__ a, const E *__restrict__ b, const E *__restrict__ g,
                            const float *initial, const float *seg_in,
                            float *__restrict__ seg_out, float *__restrict__ seg_total,
                            float *__restrict__ snap, float *fin, int H,
                            const __grid_constant__ GatedTable tab) {
    constexpr int C = GatedSimt::C, VS = GatedSimt::VS, NS = D / VS, R = D / 32;
    extern __shared__ __align__(16) float simt_sm[];
    __shared__ double sG[2][C];
    const int tid = threadIdx.x;
    const int vs = blockIdx.x % NS, h = (blockIdx.x / NS) % H, sg = blockIdx.x / (NS * H);
    int rank, s, start, len, sid;
    tab.seg(sg, rank, s);
    tab.seqs.get(rank, start, len, sid);
    const int nb = (len + C - 1) / C, ns = tab.num_segs(rank);
    const int b0 = s * tab.seg_blocks, n = max(0, min(nb, b0 + tab.seg_blocks) - b0);
    const int x0 = (tid >> 3) * R, y0 = (tid & 7) * 4;  // this thread's rows and columns
    auto tile_a = [&](int t) { return simt_sm + (t & 1) * GatedStateSimt<D>::A; };
    auto tile_b = [&](int t) { return simt_sm + 2 * GatedStateSimt<D>::A + (t & 1) * GatedStateSimt<D>::B; };
    auto block_of = [&](int t) { return REV ? b0 + n - 1 - t : b0 + t; };
    auto load = [&](int t) {
        const int row0 = start + block_of(t) * C, nv = min(C, len - block_of(t) * C);
        float *sa = tile_a(t), *sb = tile_b(t);
#pragma unroll
        for (int i = tid; i < C * D / 4; i += GatedSimt::THREADS) {
            const int rr = i / (D / 4), d = 4 * (i % (D / 4));
            simt_load4(sa + rr * D + d, a + ((size_t)(row0 + min(rr, nv - 1)) * H + h) * D + d, rr < nv);
        }
#pragma unroll
        for (int i = tid; i < C * VS / 4; i += GatedSimt::THREADS) {
            const int rr = i / (VS / 4), d = 4 * (i % (VS / 4));
            simt_load4(sb + rr * VS + d, b + ((size_t)(row0 + min(rr, nv - 1)) * H + h) * D + vs * VS + d, rr < nv);
        }
        cp_async_commit();
    };
    const bool adds = tid < GatedSimt::THREADS;  // the last warp: gate sums of the next block
    next_may_start();
    previous_done();
    auto sums = [&](int t) {
        const int blk = block_of(t);
        simt_gate_sums(sG[t & 1], g, start + blk * C, min(C, len - blk * C), H, h);
    };

    if (n > 0) {
        if (adds)
            load(0);
        else
            sums(0);
    }
    float4 X[R];
    const float *from = nullptr;
    if (seg_in != nullptr)
        from = seg_in + ((size_t)sg * H + h) * D * D;
    else if (initial != nullptr)
        from = initial + ((size_t)sid * H + h) * D * D;
#pragma unroll
    for (int r = 0; r < R; ++r)
        X[r] = from != nullptr && adds
                   ? *reinterpret_cast<const float4 *>(from + (size_t)(x0 + r) * D + vs * VS + y0)
                   : make_float4(0.f, 0.f, 0.f, 0.f);
    double total = 0.0;
    for (int t = 0; t < n; ++t) {
        const int blk = block_of(t);
        if (t + 1 < n && adds) {
            load(t + 1);
            cp_async_wait<1>();
        } else {
            cp_async_wait<0>();
        }
        __syncthreads();
        if (!adds) {  // (meets the others at the block's three barriers)
            total += sG[t & 1][C - 1];
            if (t + 1 < n) sums(t + 1);
            __syncthreads();
            __syncthreads();
            continue;
        }
        const double *G = sG[t & 1];
        float *sa = tile_a(t), *sb = tile_b(t);
#pragma unroll
        for (int i = tid; i < C * VS / 4; i += GatedSimt::THREADS) {
            const int rr = i / (VS / 4);
            const float w = expf((float)(REV ? G[rr] : G[C - 1] - G[rr]));
            float4 x = reinterpret_cast<float4 *>(sb)[i];
            reinterpret_cast<float4 *>(sb)[i] = make_float4(w * x.x, w * x.y, w * x.z, w * x.w);
        }
        if (snap != nullptr) {
            float *dst = snap + ((size_t)(tab.first_block(rank) + blk) * H + h) * D * D;
#pragma unroll
            for (int r = 0; r < R; ++r)
                *reinterpret_cast<float4 *>(dst + (size_t)(x0 + r) * D + vs * VS + y0) = X[r];
        }
        const double block_sum = G[C - 1];
        total += block_sum;
        __syncthreads();
        const float decay = expf((float)block_sum);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            X[r].x *= decay;
            X[r].y *= decay;
            X[r].z *= decay;
            X[r].w *= decay;
        }
        const int seen = min(C, (len - blk * C + 7) & ~7);  // (rows behind the sequence are zeros)
#pragma unroll 8
        for (int c = 0; c < seen; ++c) {
            const float4 bb = *reinterpret_cast<const float4 *>(sb + c * VS + y0);
            float aa[R];
            if constexpr (R == 4)
                *reinterpret_cast<float4 *>(aa) = *reinterpret_cast<const float4 *>(sa + c * D + x0);
            else
                *reinterpret_cast<float2 *>(aa) = *reinterpret_cast<const float2 *>(sa + c * D + x0);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                X[r].x = fmaf(aa[r], bb.x, X[r].x);
                X[r].y = fmaf(aa[r], bb.y, X[r].y);
                X[r].z = fmaf(aa[r], bb.z, X[r].z);
                X[r].w = fmaf(aa[r], bb.w, X[r].w);
            }
        }
        __syncthreads();  // this block's tiles may be written again
    }
    float *to = nullptr;
    if (seg_out != nullptr)
        to = seg_out + ((size_t)sg * H + h) * D * D;
    else if (fin != nullptr && s == (REV ? 0 : ns - 1))
        to = fin + ((size_t)sid * H + h) * D * D;
    if (to != nullptr && adds) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            *reinterpret_cast<float4 *>(to + (size_t)(x0 + r) * D + vs * VS + y0) = X[r];
    }
    if (seg_out != nullptr && vs == 0 && tid == 0) seg_total[(size_t)sg * H + h] = (float)total;
}

// Shared-memory tiles of the block kernels: rows of D + 4 floats (a 16-byte shift per row,
// so that eight lanes reading eight rows at one column meet eight different bank groups).
template <int D>
struct GatedSimtTiles {
    static constexpr int LD = D + 4, LP = GatedSimt::C + 4;
    static constexpr int TILE = GatedSimt::C * LD, PT = GatedSimt::C * LP;
    static constexpr int SROWS = 32, ST = SROWS * LD;  // a slab of the state
    static constexpr int FWD_BYTES = (3 * TILE + PT + ST) * 4 + GatedSimt::C * 8;
    static constexpr int BWD_BYTES = (4 * TILE + 2 * PT + ST) * 4 + GatedSimt::C * 8 + 6 * GatedSimt::C * 4 + 64;
};

// A tile; rows behind the sequence are zeros.
template <int D, typename E>
__device__ __forceinline__ void simt_load_tile(float *dst, const E *__restrict__ src, int row0, int nv, int H,
                                               int h) {
    constexpr int LD = GatedSimtTiles<D>::LD;
#pragma unroll
    for (int i = threadIdx.x; i < GatedSimt::C * D / 4; i += GatedSimt::THREADS) {
        const int r = i / (D / 4), d = 4 * (i % (D / 4));
        simt_load4(dst + r * LD + d, src + ((size_t)(row0 + min(r, nv - 1)) * H + h) * D + d, r < nv);
    }
}

// acc[r][c] += sum_d A[4 ty + r][d] B[tx + 16 c][d]: the 64 x 64 products of two tiles' rows.
template <int D>
__device__ __forceinline__ void simt_rows_by_rows(float (&acc)[4][4], const float *A, const float *B, int nv) {
    constexpr int LD = GatedSimtTiles<D>::LD;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    if (4 * ty >= nv) return;  // rows behind the sequence
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) a[r] = *reinterpret_cast<const float4 *>(A + (4 * ty + r) * LD + d);
#pragma unroll
        for (int c = 0; c < 4; ++c) b[c] = *reinterpret_cast<const float4 *>(B + (tx + 16 * c) * LD + d);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                acc[r][c] = fmaf(a[r].x, b[c].x, acc[r][c]);
                acc[r][c] = fmaf(a[r].y, b[c].y, acc[r][c]);
                acc[r][c] = fmaf(a[r].z, b[c].z, acc[r][c]);
                acc[r][c] = fmaf(a[r].w, b[c].w, acc[r][c]);
            }
    }
}

// acc[r][4 g + e] += sum_{c < n} A(4 ty + r, c) B[c][64 g + 4 tx + e].  A(i, c) = A[i * la + c],
// or A[c * la + i] with TA.  Rows i from nv on are left as they are.
template <int D, bool TA>
__device__ __forceinline__ void simt_rows_by_cols(float (&acc)[4][D / 16], const float *A, int la,
                                                  const float *B, int n, int nv) {
    constexpr int LD = GatedSimtTiles<D>::LD;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    if (4 * ty >= nv) return;
    for (int c0 = 0; c0 < n; c0 += 4) {
        float a[4][4];  // a[c][r]
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float4 f = TA ? *reinterpret_cast<const float4 *>(A + (c0 + x) * la + 4 * ty)
                                : *reinterpret_cast<const float4 *>(A + (4 * ty + x) * la + c0);
            if (TA) {
                a[x][0] = f.x, a[x][1] = f.y, a[x][2] = f.z, a[x][3] = f.w;
            } else {
                a[0][x] = f.x, a[1][x] = f.y, a[2][x] = f.z, a[3][x] = f.w;
            }
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int gq = 0; gq < D / 64; ++gq) {
                const float4 b = *reinterpret_cast<const float4 *>(B + (c0 + x) * LD + 64 * gq + 4 * tx);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    acc[r][4 * gq + 0] = fmaf(a[x][r], b.x, acc[r][4 * gq + 0]);
                    acc[r][4 * gq + 1] = fmaf(a[x][r], b.y, acc[r][4 * gq + 1]);
                    acc[r][4 * gq + 2] = fmaf(a[x][r], b.z, acc[r][4 * gq + 2]);
                    acc[r][4 * gq + 3] = fmaf(a[x][r], b.w, acc[r][4 * gq + 3]);
                }
            }
    }
}

// acc += A M (or A M^T with TM) for the D x D state M in global memory, a slab of 32
// contracted rows at a time through shared memory; the next slab is in registers meanwhile.
template <int D, bool TM>
__device__ __forceinline__ void simt_rows_by_state(float (&acc)[4][D / 16], const float *A,
                                                   const float *M, float *slab, int nv) {
    constexpr int LD = GatedSimtTiles<D>::LD, SR = GatedSimtTiles<D>::SROWS;
    constexpr int N = SR * D / 4 / GatedSimt::THREADS;
    const int tid = threadIdx.x;
    float4 x[N];
    auto fetch = [&](int c0) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int i = tid + e * GatedSimt::THREADS;
            // TM: lane -> row of M, so that the transposed stores of a warp are consecutive
            x[e] = TM ? *reinterpret_cast<const float4 *>(M + (size_t)(i % D) * D + c0 + 4 * (i / D))
                      : *reinterpret_cast<const float4 *>(M + (size_t)(c0 + i / (D / 4)) * D + 4 * (i % (D / 4)));
        }
    };
    fetch(0);
    for (int c0 = 0; c0 < D; c0 += SR) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int i = tid + e * GatedSimt::THREADS;
            if (TM) {  // slab[c][row] = M[row][c0 + c]
                float *to = slab + 4 * (i / D) * LD + i % D;
                to[0] = x[e].x, to[LD] = x[e].y, to[2 * LD] = x[e].z, to[3 * LD] = x[e].w;
            } else {
                *reinterpret_cast<float4 *>(slab + (i / (D / 4)) * LD + 4 * (i % (D / 4))) = x[e];
            }
        }
        __syncthreads();
        if (c0 + SR < D) fetch(c0 + SR);
        simt_rows_by_cols<D, false>(acc, A + c0, LD, slab, SR, nv);
    }
}

template <int D, typename E>
__device__ __forceinline__ void simt_store_rows(E *__restrict__ dst, const float (&acc)[4][D / 16], int row0,
                                                int nv, int H, int h) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (4 * ty + r < nv)
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
                simt_store4(dst + ((size_t)(row0 + 4 * ty + r) * H + h) * D + 64 * x + 4 * tx, acc[r][4 * x],
                            acc[r][4 * x + 1], acc[r][4 * x + 2], acc[r][4 * x + 3]);
}

// Output of one block of one head, from the state at its start (snap; nullptr: zero).
template <int D>
__global__ void __launch_bounds__(GatedSimt::THREADS)
    gated_prefill_simt_kernel(const float *__restrict__ q, const float *__restrict__ k, const float *__restrict__ v,
                              const float *__restrict__ g, float *__restrict__ o, const float *snap,
                              int H, const __grid_constant__ GatedTable tab) {
    using L = GatedSimtTiles<D>;
    constexpr int C = GatedSimt::C;
    extern __shared__ __align__(16) float simt_sm[];
    float *sQ = simt_sm, *sK = sQ + L::TILE, *sV = sK + L::TILE, *sP = sV + L::TILE, *slab = sP + L::PT;
    double *sG = reinterpret_cast<double *>(slab + L::ST);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int h = blockIdx.x % H, x = blockIdx.x / H;
    int rank, blk, start, len, sid;
    tab.block(x, rank, blk);
    tab.seqs.get(rank, start, len, sid);
    const int row0 = start + blk * C, nv = min(C, len - blk * C);
    previous_done();
    simt_load_tile<D>(sQ, q, row0, nv, H, h);
    simt_load_tile<D>(sK, k, row0, nv, H, h);
    simt_load_tile<D>(sV, v, row0, nv, H, h);
    cp_async_commit();
    if (threadIdx.x < 32) simt_gate_sums(sG, g, row0, nv, H, h);
    cp_async_wait<0>();
    __syncthreads();
    {
        float p[4][4] = {};
        simt_rows_by_rows<D>(p, sQ, sK, C);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int i = 4 * ty + r, j = tx + 16 * c;
                sP[i * L::LP + j] = j <= i ? p[r][c] * expf((float)(sG[i] - sG[j])) : 0.f;
            }
    }
    float acc[4][D / 16] = {};
    if (snap != nullptr) {
        simt_rows_by_state<D, false>(acc, sQ, snap + ((size_t)x * H + h) * D * D, slab, C);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float w = expf((float)sG[4 * ty + r]);
#pragma unroll
            for (int e = 0; e < D / 16; ++e) acc[r][e] *= w;
        }
    }
    __syncthreads();
    simt_rows_by_cols<D, false>(acc, sP, L::LP, sV, C, C);
    simt_store_rows<D>(o, acc, row0, nv, H, h);
}

// Sum over the 16 threads of a half-warp (the threads of one ty).
__device__ __forceinline__ float half_warp_sum(float x) {
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// Gradients of one block of one head, from the state at its start (snap) and the state's
// gradient at its end (dsnap); either may be nullptr for zero.  Bound by FMA issue and the
// shared-memory loads that feed it; a call of 1000 tokens of 4 heads, D = 64, takes 45 us, about
// half of it here.  `by_seq`: sequences of one block, whose states are the call's own (indexed
// by sequence, not by block).
template <int D, typename E>
__global__ void __launch_bounds__(GatedSimt::THREADS)
    gated_backward_simt_kernel(const E *__restrict__ q, const E *__restrict__ k, const E *__restrict__ v,
                               const E *__restrict__ g, const E *__restrict__ dout, E *__restrict__ dq,
                               E *__restrict__ dk, E *__restrict__ dv, E *__restrict__ dg,
                               const float *snap, const float *dsnap, int by_seq, int H,
                               const __grid_constant__ GatedTable tab) {
    using L = GatedSimtTiles<D>;
    constexpr int C = GatedSimt::C;
    extern __shared__ __align__(16) float simt_sm[];
    float *sQ = simt_sm, *sK = sQ + L::TILE, *sV = sK + L::TILE, *sO = sV + L::TILE;
    float *sP = sO + L::TILE, *sdP = sP + L::PT, *slab = sdP + L::PT;
    double *sG = reinterpret_cast<double *>(slab + L::ST);
    float *sR = reinterpret_cast<float *>(sG + C);  // q_i . (e^{G_i} S do_i)
    float *sE = sR + C;                             // k_j . (e^{G_C - G_j} dS v_j)
    float *sRow = sE + C;                           // sum_{j < i} W_ij
    float *sCol = sRow + C;                         // sum_{i > j} W_ij
    float *red = sCol + C;                          // 8 warps' parts of <dS, S>
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int h = blockIdx.x % H, x = blockIdx.x / H;
    int rank, blk, start, len, sid;
    tab.block(x, rank, blk);
    tab.seqs.get(rank, start, len, sid);
    const int row0 = start + blk * C, nv = min(C, len - blk * C);
    const size_t at = ((size_t)(by_seq ? sid : x) * H + h) * D * D;
    const float *S = snap != nullptr ? snap + at : nullptr, *dS = dsnap != nullptr ? dsnap + at : nullptr;
    previous_done();
    simt_load_tile<D>(sQ, q, row0, nv, H, h);
    simt_load_tile<D>(sK, k, row0, nv, H, h);
    simt_load_tile<D>(sV, v, row0, nv, H, h);
    simt_load_tile<D>(sO, dout, row0, nv, H, h);
    cp_async_commit();
    if (tid < 32) simt_gate_sums(sG, g, row0, nv, H, h);
    cp_async_wait<0>();
    __syncthreads();
    float wrow[4], wcol[4];  // e^{G_i}, e^{G_C - G_j} of this thread's rows
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        wrow[r] = expf((float)sG[4 * ty + r]);
        wcol[r] = expf((float)(sG[C - 1] - sG[4 * ty + r]));
    }
    {
        float p[4][4] = {}, dp[4][4] = {};
        simt_rows_by_rows<D>(p, sQ, sK, nv);
        simt_rows_by_rows<D>(dp, sO, sV, nv);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float row = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int i = 4 * ty + r, j = tx + 16 * c;
                const float w = j <= i ? expf((float)(sG[i] - sG[j])) : 0.f;
                const float P = j <= i ? p[r][c] * w : 0.f;
                sP[i * L::LP + j] = P;
                sdP[i * L::LP + j] = j <= i ? dp[r][c] * w : 0.f;
                p[r][c] = j < i ? P * dp[r][c] : 0.f;  // W_ij of the pairs j < i
                row += p[r][c];
            }
            row = half_warp_sum(row);
            if (tx == 0) sRow[4 * ty + r] = row;
        }
        // column sums of W: this thread's four rows, then the 16 row groups through the slab
#pragma unroll
        for (int c = 0; c < 4; ++c) slab[ty * C + tx + 16 * c] = p[0][c] + p[1][c] + p[2][c] + p[3][c];
    }
    __syncthreads();
    if (tid < C) {
        float col = 0.f;
        for (int y = 0; y < 16; ++y) col += slab[y * C + tid];
        sCol[tid] = col;
    }
    // dq = dP k + e^{G_i} S do_i
    float acc[4][D / 16] = {};
    if (S != nullptr) simt_rows_by_state<D, true>(acc, sO, S, slab, nv);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < D / 16; ++e) {
            acc[r][e] *= wrow[r];
            s = fmaf(acc[r][e], sQ[(4 * ty + r) * L::LD + 64 * (e / 4) + 4 * tx + (e & 3)], s);
        }
        s = half_warp_sum(s);
        if (tx == 0) sR[4 * ty + r] = s;
    }
    __syncthreads();
    simt_rows_by_cols<D, false>(acc, sdP, L::LP, sK, (nv + 3) & ~3, nv);
    simt_store_rows<D>(dq, acc, row0, nv, H, h);
    // dk = dP^T q + e^{G_C - G_j} dS v_j
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < D / 16; ++e) acc[r][e] = 0.f;
    if (dS != nullptr) simt_rows_by_state<D, true>(acc, sV, dS, slab, nv);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < D / 16; ++e) {
            acc[r][e] *= wcol[r];
            s = fmaf(acc[r][e], sK[(4 * ty + r) * L::LD + 64 * (e / 4) + 4 * tx + (e & 3)], s);
        }
        s = half_warp_sum(s);
        if (tx == 0) sE[4 * ty + r] = s;
    }
    simt_rows_by_cols<D, true>(acc, sdP, L::LP, sQ, (nv + 3) & ~3, nv);
    simt_store_rows<D>(dk, acc, row0, nv, H, h);
    // dv = P^T do + e^{G_C - G_j} dS^T k_j
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < D / 16; ++e) acc[r][e] = 0.f;
    if (dS != nullptr) simt_rows_by_state<D, false>(acc, sK, dS, slab, nv);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < D / 16; ++e) acc[r][e] *= wcol[r];
    simt_rows_by_cols<D, true>(acc, sP, L::LP, sO, (nv + 3) & ~3, nv);
    simt_store_rows<D>(dv, acc, row0, nv, H, h);
    // <dS, S>
    float f = 0.f;
    if (S != nullptr && dS != nullptr)
        for (int i = tid; i < D * D; i += GatedSimt::THREADS) f = fmaf(S[i], dS[i], f);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) f += __shfl_xor_sync(0xffffffffu, f, off);
    if ((tid & 31) == 0) red[tid >> 5] = f;
    __syncthreads();
    if (tid < 32 && dg != nullptr) {
        // dg_t = e^{G_C} <dS, S> + sum_{i >= t} sR_i + sum_{j < t} (sE_j + sCol_j - sRow_j):
        // sum_{j < t <= i} W_ij grows from t to t + 1 by the pairs that begin at t and loses
        // those that end there.  Two tokens per lane.
        float through = 0.f;
        for (int w = 0; w < 8; ++w) through += red[w];
        through *= expf((float)sG[C - 1]);
        const int t0 = 2 * tid;
        const float r0 = sR[t0], r1 = sR[t0 + 1];
        const float e0 = sE[t0] + sCol[t0] - sRow[t0], e1 = sE[t0 + 1] + sCol[t0 + 1] - sRow[t0 + 1];
        float up = r0 + r1, down = e0 + e1;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const float a = __shfl_down_sync(0xffffffffu, up, off), b = __shfl_up_sync(0xffffffffu, down, off);
            if (tid + off < 32) up += a;
            if (tid >= off) down += b;
        }
        // up: sum_{i >= t0}; down: sum_{j <= t0 + 1}
        float before = __shfl_up_sync(0xffffffffu, down, 1);  // sum_{j < t0}
        if (tid == 0) before = 0.f;
        float after = __shfl_down_sync(0xffffffffu, up, 1);   // sum_{i >= t0 + 2}
        if (tid == 31) after = 0.f;
        if (t0 < nv) dg[(size_t)(row0 + t0) * H + h] = from_f32<E>(through + up + before);
        if (t0 + 1 < nv) dg[(size_t)(row0 + t0 + 1) * H + h] = from_f32<E>(through + after + r1 + before + e0);
    }
}

// ------------------------------------------------------------------ one token
// state_out <- e^g state_in + k v^T, o = state_out^T q for one token of one head, by 256
// threads.  Without state_in the state before was zero; without state_out it is not kept
// (BOTH: both are there, which spares a full batch 1.5 % of its time).
template <int D, typename T, bool BOTH>
__device__ __forceinline__ void gated_one_token(const T *__restrict__ q, const T *__restrict__ k,
                                                const T *__restrict__ v, const T *__restrict__ g, T *__restrict__ o,
                                                const float4 *state_in, float4 *state_out) {
    constexpr int C4 = D / 4, RG = 256 / C4, RPT = D / RG;
    __shared__ float sq[D], sk[D];
    __shared__ float red[RG][D];
    const int tid = threadIdx.x, c4 = tid % C4, rg = tid / C4;
    float4 x[RPT];
#pragma unroll
    for (int t = 0; t < RPT; ++t)
        x[t] = BOTH || state_in != nullptr ? __ldcs(&state_in[(size_t)(rg + RG * t) * C4 + c4])
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
    if (tid < D) {
        sq[tid] = to_f32(q[tid]);
        sk[tid] = to_f32(k[tid]);
    }
    const float a = g != nullptr ? expf(clamp_gate(to_f32(*g))) : 1.f;
    const float v0 = to_f32(v[4 * c4]), v1 = to_f32(v[4 * c4 + 1]), v2 = to_f32(v[4 * c4 + 2]),
                v3 = to_f32(v[4 * c4 + 3]);
    __syncthreads();
    float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
    for (int t = 0; t < RPT; ++t) {
        const int r = rg + RG * t;
        const float kr = sk[r], qr = sq[r];
        x[t].x = fmaf(kr, v0, a * x[t].x);
        x[t].y = fmaf(kr, v1, a * x[t].y);
        x[t].z = fmaf(kr, v2, a * x[t].z);
        x[t].w = fmaf(kr, v3, a * x[t].w);
        if (BOTH || state_out != nullptr) __stcs(&state_out[(size_t)r * C4 + c4], x[t]);
        a0 = fmaf(qr, x[t].x, a0);
        a1 = fmaf(qr, x[t].y, a1);
        a2 = fmaf(qr, x[t].z, a2);
        a3 = fmaf(qr, x[t].w, a3);
    }
    red[rg][4 * c4 + 0] = a0;
    red[rg][4 * c4 + 1] = a1;
    red[rg][4 * c4 + 2] = a2;
    red[rg][4 * c4 + 3] = a3;
    __syncthreads();
    if (tid < D) {
        float out = 0.f;
#pragma unroll
        for (int y = 0; y < RG; ++y) out += red[y][tid];
        o[tid] = from_f32<T>(out);
    }
}

// One token per row, the state in slot slots[b] of a pool of num_slots (row b itself without
// slots), updated in place.  One CTA of 256 threads per
// (row, head), as the plain decode step: HBM-bound, 8 D^2 bytes against 6 D^2 flops (256 rows,
// 64 heads, D = 128: 335 us, 6.5 TB/s; one row 3.5 us).
// A row of slot -1 is padding: nothing of it is read or written.  A slot outside the pool,
// or one that an earlier row of the batch has (two rows would race for one state), is
// skipped in the same way and recorded as DEV_RANGE.
template <int D, typename T>
__global__ void __launch_bounds__(256)
    gated_decode_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                        const T *__restrict__ g, float *state, T *__restrict__ o, int H,
                        const int *__restrict__ slots, int num_slots) {
    const int b = blockIdx.x / H, h = blockIdx.x % H, tid = threadIdx.x;
    const size_t vec = (size_t)blockIdx.x * D;
    int slot = b;
    if (slots != nullptr) {
        slot = slots[b];
        int bad = 0;
        if (slot >= 0 && slot < num_slots) {
            for (int i = tid; i < b; i += 256) bad |= slots[i] == slot;
        } else {
            bad = 1;
        }
        if (__syncthreads_or(bad)) {
            if (tid == 0 && slot != -1) record_fault(DEV_RANGE);
            return;
        }
    }
    float4 *S = reinterpret_cast<float4 *>(state + ((size_t)slot * H + h) * D * D);
    gated_one_token<D, T, true>(q + vec, k + vec, v + vec, g != nullptr ? g + blockIdx.x : nullptr, o + vec, S, S);
}

// The sequences of one token of a packed call, rows of the packed arrays in place: the
// state from the sequence's initial state (or zero) to its final state (or nowhere).  256 of
// them, 64 heads, D = 128, take 318 us here; as blocks of the prefill kernel they took 1844.
template <int D, typename T>
__global__ void __launch_bounds__(256)
    gated_rows_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                      const T *__restrict__ g, T *__restrict__ o, const float *initial, float *fin, int H,
                      const __grid_constant__ OneTokenTable tab) {
    const int i = blockIdx.x / H, h = blockIdx.x % H;
    const size_t row = (size_t)(tab.identity ? i : tab.row[i]) * H + h;
    const size_t state = ((size_t)(tab.identity ? i : tab.sid[i]) * H + h) * D * D;
    gated_one_token<D, T, false>(q + row * D, k + row * D, v + row * D, g != nullptr ? g + row : nullptr, o + row * D,
                                 initial != nullptr ? reinterpret_cast<const float4 *>(initial + state) : nullptr,
                                 fin != nullptr ? reinterpret_cast<float4 *>(fin + state) : nullptr);
}

}  // namespace la
