// Selective scan for serving: packed prompts of different lengths, and single tokens, on a pool of
// states (include/ssm_scan.h).
//
//     h_t = exp(delta_t A) h_{t-1} + w_t B_t x_t,   y_t = (C_t . h_t + D x_t) [z_t sigmoid(z_t)],
//     w = delta (Euler) or (exp(delta A) - 1) / A (zero-order hold).
//
// Prompts.  One exp2 a state and step bounds them from below (16 lanes a cycle and SM, so 8 cycles a warp
// instruction); next come shared memory (B, C, delta for every lane: one wavefront a cycle and SM)
// and the issue slots.  Memory traffic, 8 bytes a channel and step in bf16, is a small share.  The
// recurrence itself is short, but serial, and everything else is not.  So a CTA takes a few channels of one
// whole sequence, and its warps take turns of U steps in a ring: a warp loads its turn one round
// ahead, computes transitions and input terms of all U steps, then waits for the state from the warp
// before, runs its U steps, hands the state on through shared memory and a named barrier, and finishes its y's
// while the others go on.  A sequence of any length is one pass: nothing is evaluated twice, no segment
// summaries, no workspace, and no split to choose.  (Measured before: time segments
// with summaries and a carry, which evaluate every exp2 twice: 4096 steps of 1536 channels took 98 us
// against 86, a ragged batch of 24 prompts on 4096 channels 445 us against 325.)
//
// Single tokens.  Bound by the states' traffic, 8 N bytes a channel and row.
#include "layer_common.cuh"
#include "real_common.cuh"

namespace ssm {
namespace serve {
namespace {

using real::ex2_pair;
using real::f2;
using real::kFull;

// four B or C elements of a row, as fp32
template <typename E>
__device__ __forceinline__ float4 quad_f4(const typename Vec<E, 4>::Raw& r) {
    float2 o[2];
    Vec<E, 4>::unpack(r, o);
    return make_float4(o[0].x, o[0].y, o[1].x, o[1].y);
}

// A log2(e) of a pair of states, finite even where exp(A_log) is not: there a step of any length still leaves
// nothing of the state, but a step of length zero (past the end of a sequence, inside its last turn) all of it.
// A NaN stays.
__device__ __forceinline__ float2 rate_pair(float l0, float l1) {
    const float a = expf(l0) * kLog2e, b = expf(l1) * kLog2e, top = 3.402823466e38f;
    return make_float2(a > top ? -top : -a, b > top ? -top : -b);
}

// w B x for a pair of states: delta and delta x (each twice), e = exp(delta A), A2 = A log2(e), Ar = 1 / A
template <bool ZOH>
__device__ __forceinline__ float2 input_term(float2 dlt, float2 dx, float2 e, float2 A2, float2 Ar, float2 bq) {
    if constexpr (ZOH) {
        const float2 z = __fmul2_rn(__fmul2_rn(dlt, A2), f2(kLn2));
        const float2 rz = __fmul2_rn(f2(rcp_mufu(dlt.x)), Ar);
        return __fmul2_rn(__fmul2_rn(dx, real::zoh_e1(z, e, rz)), bq);
    } else {
        return __fmul2_rn(dx, bq);
    }
}

// softplus_fast of a pair in packed arithmetic.
__device__ __forceinline__ float2 softplus_pair(float2 v) {
    const float2 z = __fmul2_rn(make_float2(fabsf(v.x), fabsf(v.y)), f2(-kLog2e));
    const float2 e = ex2_pair(z), a = __fadd2_rn(e, f2(2.0f));
    const float2 s = __fmul2_rn(e, make_float2(rcp_mufu(a.x), rcp_mufu(a.y))), w = __fmul2_rn(s, s);
    float2 q = __ffma2_rn(w, f2(0.28011780977249146f), f2(0.2800184488296509f));
    q = __ffma2_rn(w, q, f2(0.4002152383327484f));
    q = __ffma2_rn(w, q, f2(0.666664183139801f));
    q = __ffma2_rn(w, q, f2(2.0f));
    return __ffma2_rn(s, q, make_float2(fmaxf(v.x, 0.0f), fmaxf(v.y, 0.0f)));
}

// Prompts.  A lane owns four states of two neighbouring channels: NG = N / 4 lanes a pair of channels, CW
// channels a CTA.  Each of its NW warps holds all of them, for its turns of U steps.  Row by row a lane
// holds SH of a turn's steps, the same ones whose sums the reduction over the NG lanes leaves in it.
// Two forms, chosen by prompt_impl:
//   MANY: turns of four steps, four warps a CTA, four CTAs an SM, which share it.
//   Few: turns of eight steps, eight warps and one CTA an SM, so that a step's share of the hand-over is small.
//   With N = 16 a turn is also reduced to h_out = P h_in + S before the state arrives (kWhole): more
//   arithmetic, but only one product on the chain from warp to warp (one sequence of 3000 steps on 4096 channels
//   145 -> 127 us; with N = 8 the arithmetic costs what the chain gains, with N = 4 more: 92 against 132).
template <int N, bool MANY>
struct PromptCfg {
    static constexpr int NG = N / 4;
    static constexpr int CW = 64 / NG;
    static constexpr int U = MANY ? 4 : 8;
    static constexpr int NW = MANY ? 4 : 8;
    static constexpr int SH = U / NG;
    static constexpr int kCtas = MANY ? 4 : 1;   // an SM
    static constexpr bool kWhole = !MANY && N == 16;
};

// A pair of neighbouring channels as it lies in a row.
template <typename E> struct Pair;
template <> struct Pair<float> {
    using Raw = float2;
    static __device__ __forceinline__ float2 to_f(Raw r) { return r; }
    static __device__ __forceinline__ Raw from_f(float2 v) { return v; }
};
template <> struct Pair<__nv_bfloat16> {
    using Raw = unsigned;
    static __device__ __forceinline__ float2 to_f(Raw r) { return bf16_pair(r); }
    static __device__ __forceinline__ Raw from_f(float2 v) { return pack_bf16(v); }
};

// Hand-over between two warps: named barriers 1 .. NW, one per receiving warp.
__device__ __forceinline__ void hand_wait(int w) { asm volatile("bar.sync %0, 64;" ::"r"(w + 1) : "memory"); }
__device__ __forceinline__ void hand_over(int w) { asm volatile("bar.arrive %0, 64;" ::"r"(w + 1) : "memory"); }

template <typename E, int N, bool ZOH, bool MANY>
__global__ void __launch_bounds__(PromptCfg<N, MANY>::NW * 32, PromptCfg<N, MANY>::kCtas)
scan_prompt_kernel(ScanServeArgs a) {
    using Cfg = PromptCfg<N, MANY>;
    constexpr bool WHOLE = Cfg::kWhole;
    using PR = typename Pair<E>::Raw;
    using BR = typename Vec<E, 4>::Raw;
    constexpr int NG = Cfg::NG, CW = Cfg::CW, U = Cfg::U, SH = Cfg::SH, NP = CW / 2, NW = Cfg::NW;
    __shared__ float2 s_dlt[NW][U][NP];         // delta and delta x of a pair of channels
    __shared__ float2 s_dx[NW][U][NP];
    __shared__ __align__(16) BR s_b[NW][U * NG], s_c[NW][U * NG];  // four states of a step, as loaded
    __shared__ float4 s_h[NW][2][32];
    __shared__ int s_seq;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ng = lane % NG, dl = lane / NG;
    const int d = (int)(blockIdx.x % a.ndt) * CW + 2 * dl, n0 = ng * 4;  // the lane's channels d, d + 1
    const bool dv = d < a.D;
    const int dc = dv ? d : 0;  // lanes past the last channel run along on channel 0 and store nothing

    float4 l[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) l[c] = __ldg(reinterpret_cast<const float4*>(a.A_log + (size_t)(dc + c) * N + n0));
    if (a.status && blockIdx.x == 0)
        check_batch(a.offsets, a.slot, a.S, a.rows, a.slots, a.max_len, a.status);
    const int rank = (int)(blockIdx.x / a.ndt);
    int s = rank;
    if (a.sorted) {  // the longest sequences first
        const int j = threadIdx.x;
        if (j < a.S) {
            const int len = length_of(a.offsets, j);
            int r = 0;
            for (int i = 0; i < a.S; ++i) {
                const int other = length_of(a.offsets, i);
                r += other > len || (other == len && i < j);
            }
            if (r == rank) s_seq = j;
        }
        __syncthreads();
        s = s_seq;
    }
    const Span sp = seq_span(a.offsets, a.slot, s, a.rows, a.slots, a.max_len);
    if (!sp.ok) return;  // the whole CTA
    const int n = sp.end - sp.first, turns = (n + U - 1) / U;

    // the sequence's first row; rows are addressed by 32-bit byte strides
    const size_t r0 = (size_t)sp.first;
    const bool gated = a.z != nullptr;
    const unsigned ldx = (unsigned)(a.ldx * sizeof(E)), ldd = (unsigned)(a.ldd * sizeof(E));
    const unsigned ldz = (unsigned)(a.ldz * sizeof(E)), ldy = (unsigned)(a.ldy * sizeof(E));
    const unsigned ldb = (unsigned)(a.ldb * sizeof(E)), ldc = (unsigned)(a.ldc * sizeof(E));
    const E* px = static_cast<const E*>(a.x) + r0 * a.ldx + dc;
    const E* pd = static_cast<const E*>(a.draw) + r0 * a.ldd + dc;
    const E* pz = gated ? static_cast<const E*>(a.z) + r0 * a.ldz + dc : nullptr;
    E* py = static_cast<E*>(a.y) + r0 * a.ldy + dc;
    const int brow = lane / NG, bcol = (lane % NG) * 4;  // B and C: the first U * NG lanes
    const E* pB = static_cast<const E*>(a.Bm) + r0 * a.ldb + bcol;
    const E* pC = static_cast<const E*>(a.Cm) + r0 * a.ldc + bcol;

    PR nx[SH], nd[SH], nz[SH];
    BR nB, nC;
    auto load = [&](int t) {  // past the end: the last row again
#pragma unroll
        for (int k = 0; k < SH; ++k) {
            const int r = min(t + ng * SH + k, n - 1);
            nx[k] = *reinterpret_cast<const PR*>(row_at(px, r, ldx));
            nd[k] = *reinterpret_cast<const PR*>(row_at(pd, r, ldd));
            if (gated) nz[k] = *reinterpret_cast<const PR*>(row_at(pz, r, ldz));
        }
        if (lane < U * NG) {
            const int r = min(t + brow, n - 1);
            nB = ld_vec<E, 4>(row_at(pB, r, ldb));
            nC = ld_vec<E, 4>(row_at(pC, r, ldc));
        }
    };
    if (warp < turns) load(warp * U);
    if (__syncthreads_or(named_before(a.slot, s, sp.slot, threadIdx.x, NW * 32))) {
        if (threadIdx.x == 0) flag_if(a.status, kStatusInvalid);
        return;
    }
    float2 A2[2][2], Ar[2][2];  // [channel][pair of states]
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        A2[c][0] = rate_pair(l[c].x, l[c].y);
        A2[c][1] = rate_pair(l[c].z, l[c].w);
        if (ZOH) {
            Ar[c][0] = make_float2(-expf(-l[c].x), -expf(-l[c].y));
            Ar[c][1] = make_float2(-expf(-l[c].z), -expf(-l[c].w));
        }
    }
    const float2 dsk = *reinterpret_cast<const float2*>(a.Dskip + dc);
    float* entry = sp.slot >= 0 && dv ? a.pool + ((size_t)sp.slot * a.D + d) * N + n0 : nullptr;
    float4 h4[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    if (warp == 0 && entry) {
        if (a.carry && a.carry[s])
#pragma unroll
            for (int c = 0; c < 2; ++c) h4[c] = *reinterpret_cast<const float4*>(entry + c * N);
        if (turns == 0)
#pragma unroll
            for (int c = 0; c < 2; ++c) *reinterpret_cast<float4*>(entry + c * N) = h4[c];
    }

    for (int i = warp; i < turns; i += NW) {
        const int t = i * U;
        // delta and delta x of the turn, the steps side by side
        float2 x[SH], z[SH];
#pragma unroll
        for (int k = 0; k < SH; ++k) {
            const int u = ng * SH + k;
            x[k] = Pair<E>::to_f(nx[k]);
            if (gated) z[k] = Pair<E>::to_f(nz[k]);
            float2 dl2 = softplus_pair(Pair<E>::to_f(nd[k])), dx2 = __fmul2_rn(dl2, x[k]);
            if (t + u >= n) dl2 = dx2 = f2(0.f);  // a step that is not there changes nothing
            s_dlt[warp][u][dl] = dl2;
            s_dx[warp][u][dl] = dx2;
        }
        if (lane < U * NG) {
            s_b[warp][lane] = t + brow < n ? nB : Vec<E, 4>::zero();
            s_c[warp][lane] = t + brow < n ? nC : Vec<E, 4>::zero();
        }
        __syncwarp();
        if (i + NW < turns) load(t + NW * U);
        // transitions and input terms: nothing here waits for the state
        float2 e[U][2][2], w[U][2][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float2 dlt = s_dlt[warp][u][dl], dx = s_dx[warp][u][dl];
            float2 bq[2];
            Vec<E, 4>::unpack(s_b[warp][u * NG + ng], bq);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                e[u][0][p] = ex2_pair(__fmul2_rn(f2(dlt.x), A2[0][p]));
                e[u][1][p] = ex2_pair(__fmul2_rn(f2(dlt.y), A2[1][p]));
                w[u][0][p] = input_term<ZOH>(f2(dlt.x), f2(dx.x), e[u][0][p], A2[0][p], Ar[0][p], bq[p]);
                w[u][1][p] = input_term<ZOH>(f2(dlt.y), f2(dx.y), e[u][1][p], A2[1][p], Ar[1][p], bq[p]);
            }
        }
        float2 P[2][2], out[2][2];  // the turn as a whole: out = P h + out
        if (WHOLE) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    P[c][p] = e[0][c][p];
                    out[c][p] = w[0][c][p];
#pragma unroll
                    for (int u = 1; u < U; ++u) {
                        P[c][p] = __fmul2_rn(P[c][p], e[u][c][p]);
                        out[c][p] = __ffma2_rn(e[u][c][p], out[c][p], w[u][c][p]);
                    }
                }
        }
        // from the warp before
        if (i > 0) {
            hand_wait(warp);
            h4[0] = s_h[warp][0][lane];
            h4[1] = s_h[warp][1][lane];
        }
        float2 h[2][2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            h[c][0] = make_float2(h4[c].x, h4[c].y);
            h[c][1] = make_float2(h4[c].z, h4[c].w);
        }
        auto recur = [&]() {  // e[u] becomes the state at step u
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int p = 0; p < 2; ++p) h[c][p] = e[u][c][p] = __ffma2_rn(e[u][c][p], h[c][p], w[u][c][p]);
        };
        if (!WHOLE) recur();
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int p = 0; p < 2; ++p) out[c][p] = !WHOLE ? h[c][p] : __ffma2_rn(P[c][p], h[c][p], out[c][p]);
        // to the warp after
        if (i + 1 < turns) {
            const int to = warp + 1 == NW ? 0 : warp + 1;
#pragma unroll
            for (int c = 0; c < 2; ++c)
                s_h[to][c][lane] = make_float4(out[c][0].x, out[c][0].y, out[c][1].x, out[c][1].y);
            hand_over(to);
        } else {
            if (entry)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    *reinterpret_cast<float4*>(entry + c * N) =
                        make_float4(out[c][0].x, out[c][0].y, out[c][1].x, out[c][1].y);
            if (dv && !(real::all_finite<4>(out[0]) && real::all_finite<4>(out[1])))
                flag_if(a.status, kStatusNonFinite);
        }
        if (WHOLE) recur();
        // y: the lane's part of the sums over the states, then their reduction
        float yp[2 * U];  // [step][channel]
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float2 cq[2];
            Vec<E, 4>::unpack(s_c[warp][u * NG + ng], cq);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float2 acc = __ffma2_rn(cq[1], e[u][c][1], __fmul2_rn(cq[0], e[u][c][0]));
                yp[2 * u + c] = acc.x + acc.y;
            }
        }
        real::reduce_scatter<2 * U, NG>(yp, ng);
#pragma unroll
        for (int k = 0; k < SH; ++k) {
            const int r = t + ng * SH + k;
            float2 v = __ffma2_rn(dsk, x[k], make_float2(yp[2 * k], yp[2 * k + 1]));
            if (gated) v = __fmul2_rn(v, silu_pair(z[k]));
            if (dv && r < n) *reinterpret_cast<PR*>(row_at(py, r, ldy)) = Pair<E>::from_f(v);
        }
        __syncwarp();
    }
}

// ---------------------------------------------------------------- single tokens
// Four states a thread, N / 4 lanes a channel.
struct StepRow {  // what one row adds to the state
    float2 A2[2], Ar[2];
    float dsk;
};

template <bool ZOH>
__device__ __forceinline__ StepRow step_consts(float4 l, float dsk) {
    StepRow c;
    c.A2[0] = rate_pair(l.x, l.y);
    c.A2[1] = rate_pair(l.z, l.w);
    if (ZOH) {
        c.Ar[0] = make_float2(-expf(-l.x), -expf(-l.y));
        c.Ar[1] = make_float2(-expf(-l.z), -expf(-l.w));
    }
    c.dsk = dsk;
    return c;
}

// h <- exp(delta A) h + w B x; returns (the channel's) y before the gate, in every lane of the channel.
template <typename E, int NG, bool ZOH>
__device__ __forceinline__ float step_row(const StepRow& c, float2 (&h)[2], E x, E dr,
                                          typename Vec<E, 4>::Raw rB, typename Vec<E, 4>::Raw rC) {
    const float xf = Elem<E>::to_f(x);
    const float dlt = softplus_fast(Elem<E>::to_f(dr)), dx = dlt * xf;
    float2 bq[2], cq[2], acc = f2(0.f);
    Vec<E, 4>::unpack(rB, bq);
    Vec<E, 4>::unpack(rC, cq);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 e = ex2_pair(__fmul2_rn(f2(dlt), c.A2[i]));
        h[i] = __ffma2_rn(e, h[i], input_term<ZOH>(f2(dlt), f2(dx), e, c.A2[i], c.Ar[i], bq[i]));
        acc = __ffma2_rn(cq[i], h[i], acc);
    }
    float v = acc.x + acc.y;
#pragma unroll
    for (int m = 1; m < NG; m <<= 1) v += __shfl_xor_sync(kFull, v, m);
    return fmaf(c.dsk, xf, v);
}

// One row a CTA, every load in flight at once: the shortest way for few rows.
template <typename E, int N, bool ZOH>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanServeArgs a) {
    constexpr int NG = N / 4, DC = 256 / NG;
    const int tid = threadIdx.x, ng = tid % NG, dl = tid / NG, n0 = ng * 4;
    const int d = blockIdx.x * DC + dl, row = blockIdx.y;
    const bool dv = d < a.D;
    const int dc = dv ? d : 0;
    const float4 l = __ldg(reinterpret_cast<const float4*>(a.A_log + (size_t)dc * N + n0));
    const float dsk = a.Dskip[dc];
    const int k = a.slot ? a.slot[row] : row;
    const bool live = k >= 0 && k < a.slots, work = dv && live;
    typename Vec<E, 4>::Raw rB = Vec<E, 4>::zero(), rC = Vec<E, 4>::zero();
    E x = Elem<E>::from_f(0.f), dr = x, z = x;
    if (live) {  // a padding row is not read
        rB = ld_vec<E, 4>(static_cast<const E*>(a.Bm) + row * a.ldb + n0);
        rC = ld_vec<E, 4>(static_cast<const E*>(a.Cm) + row * a.ldc + n0);
        x = static_cast<const E*>(a.x)[row * a.ldx + dc];
        dr = static_cast<const E*>(a.draw)[row * a.ldd + dc];
        if (a.z) z = static_cast<const E*>(a.z)[row * a.ldz + dc];
    }
    float* entry = a.pool + ((size_t)(live ? k : 0) * a.D + dc) * N + n0;
    const float4 h4 = work ? *reinterpret_cast<const float4*>(entry) : make_float4(0.f, 0.f, 0.f, 0.f);
    const bool repeated = a.slot && __syncthreads_or(named_before(a.slot, row, live ? k : -1, tid, 256));
    if (k >= a.slots || repeated) {
        if (tid == 0 && blockIdx.x == 0) flag_if(a.status, kStatusInvalid);
        return;
    }
    const StepRow c = step_consts<ZOH>(l, dsk);
    float2 h[2] = {make_float2(h4.x, h4.y), make_float2(h4.z, h4.w)};
    float v = step_row<E, NG, ZOH>(c, h, x, dr, rB, rC);
    if (!work) return;
    *reinterpret_cast<float4*>(entry) = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
    if (!real::all_finite<4>(h)) flag_if(a.status, kStatusNonFinite);
    if (ng == 0) {
        if (a.z) v *= silu_fast(Elem<E>::to_f(z));
        static_cast<E*>(a.y)[row * a.ldy + d] = Elem<E>::from_f(v);
    }
}

// Up to kStepRows rows a CTA, in groups of four.  The states' traffic is all that should count, so each
// thread keeps the states of two groups on their way (cp.async into its own places of a ring) while it
// computes a third, and the instructions a row are kept few: A once for all rows, B and C once in fp32 in shared
// memory, softplus, gate and y of a row in one of the channel's NG lanes each (lane ng: rows ng * SH ..).
constexpr int kStepRows = 64, kStepStages = 3, kStepGroup = 4;

template <int N>
struct StepCfg {
    static constexpr int oBC = kStepStages * kStepGroup * 256 * 16;
    static constexpr int kBytes = oBC + 2 * kStepRows * N * 4;
};

template <typename E, int N, bool ZOH>
__global__ void __launch_bounds__(256, 3) scan_step_batch_kernel(ScanServeArgs a, int rows_per_cta) {
    constexpr int NG = N / 4, DC = 256 / NG, R = kStepGroup, SH = R / NG;
    extern __shared__ __align__(16) unsigned char smem[];
    float4* ring = reinterpret_cast<float4*>(smem) + threadIdx.x;  // slot i: ring[i * 256]
    float4* sB = reinterpret_cast<float4*>(smem + StepCfg<N>::oBC);  // [row][NG], then C the same
    float4* sC = sB + kStepRows * NG;
    __shared__ int s_slot[kStepRows];                              // -1: leave the row alone
    const int tid = threadIdx.x, ng = tid % NG, dl = tid / NG, n0 = ng * 4;
    const int d = blockIdx.x * DC + dl;
    const bool dv = d < a.D;
    const int dc = dv ? d : 0;
    const int row0 = blockIdx.y * rows_per_cta, nrows = min(rows_per_cta, a.rows - row0);
    const float4 l = __ldg(reinterpret_cast<const float4*>(a.A_log + (size_t)dc * N + n0));
    const float dsk = a.Dskip[dc];
    if (tid < kStepRows) {
        const int k = tid < nrows ? (a.slot ? a.slot[row0 + tid] : row0 + tid) : -1;
        if (k >= a.slots && blockIdx.x == 0) flag_if(a.status, kStatusInvalid);
        s_slot[tid] = k < a.slots ? k : -1;
    }
    __syncthreads();
    if (a.slot) {  // rows that name an entry which an earlier row names: 256 / kStepRows threads a row
        constexpr int TR = 256 / kStepRows;
        const int r = tid / TR;
        const bool hit = named_before(a.slot, row0 + r, s_slot[r], tid % TR, TR);
        __syncthreads();
        if (hit) {
            s_slot[r] = -1;
            if (blockIdx.x == 0) flag_if(a.status, kStatusInvalid);
        }
        __syncthreads();
    }
    float* pool = a.pool + (size_t)dc * N + n0;
    const unsigned entry = (unsigned)((size_t)a.D * N * sizeof(float));  // bytes; below 2^27
    auto issue = [&](int r, int stage) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int k = r + i < nrows ? s_slot[r + i] : -1;
            if (k >= 0) real::cp_async16(ring + (stage * R + i) * 256, row_at(pool, k, entry), true);
        }
        real::cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStepStages - 1; ++i) issue(i * R, i);
    // the lane's rows of a group: r + ng * SH + j
    const unsigned ldx = (unsigned)(a.ldx * sizeof(E)), ldd = (unsigned)(a.ldd * sizeof(E));
    const unsigned ldz = (unsigned)(a.ldz * sizeof(E)), ldy = (unsigned)(a.ldy * sizeof(E));
    const E* px = static_cast<const E*>(a.x) + row0 * a.ldx + dc;
    const E* pd = static_cast<const E*>(a.draw) + row0 * a.ldd + dc;
    const E* pz = a.z ? static_cast<const E*>(a.z) + row0 * a.ldz + dc : nullptr;
    E* py = static_cast<E*>(a.y) + row0 * a.ldy + dc;
    E nx[SH], nd[SH], nz[SH];
    int nk[SH];
    auto fetch = [&](int r0) {  // a padding row is not read
#pragma unroll
        for (int j = 0; j < SH; ++j) {
            const int r = r0 + ng * SH + j;
            nk[j] = r < nrows ? s_slot[r] : -1;
            nx[j] = nd[j] = nz[j] = Elem<E>::from_f(0.f);
            if (nk[j] >= 0) {
                nx[j] = *row_at(px, r, ldx);
                nd[j] = *row_at(pd, r, ldd);
                if (pz) nz[j] = *row_at(pz, r, ldz);
            }
        }
    };
    fetch(0);
    for (int i = tid; i < nrows * NG; i += 256) {
        const int r = i / NG, c = (i % NG) * 4;
        if (s_slot[r] < 0) continue;
        sB[i] = quad_f4<E>(ld_vec<E, 4>(static_cast<const E*>(a.Bm) + (row0 + r) * a.ldb + c));
        sC[i] = quad_f4<E>(ld_vec<E, 4>(static_cast<const E*>(a.Cm) + (row0 + r) * a.ldc + c));
    }
    const StepRow c = step_consts<ZOH>(l, dsk);
    float2 finite = f2(0.f);  // becomes NaN with the first infinity or NaN in a state
    __syncthreads();
    int stage = 0;
    for (int r = 0; r < nrows; r += R) {
        float dlt[SH], dx[SH], x[SH], z[SH], yp[R];
        int ky[SH];
#pragma unroll
        for (int j = 0; j < SH; ++j) {
            ky[j] = nk[j];
            x[j] = Elem<E>::to_f(nx[j]);
            z[j] = Elem<E>::to_f(nz[j]);
            dlt[j] = softplus_fast(Elem<E>::to_f(nd[j]));
            dx[j] = dlt[j] * x[j];
        }
        issue(r + (kStepStages - 1) * R, stage == 0 ? kStepStages - 1 : stage - 1);
        fetch(r + R);
        real::cp_async_wait<kStepStages - 1>();
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float di = dlt[i % SH], xi = dx[i % SH];
            if (NG > 1) {
                di = __shfl_sync(kFull, di, i / SH, NG);
                xi = __shfl_sync(kFull, xi, i / SH, NG);
            }
            yp[i] = 0.f;
            const int k = r + i < nrows ? s_slot[r + i] : -1;
            if (k < 0) continue;  // the whole CTA
            const float4 h4 = ring[(stage * R + i) * 256], b4 = sB[(r + i) * NG + ng], c4 = sC[(r + i) * NG + ng];
            const float2 bq[2] = {make_float2(b4.x, b4.y), make_float2(b4.z, b4.w)};
            const float2 cq[2] = {make_float2(c4.x, c4.y), make_float2(c4.z, c4.w)};
            float2 h[2] = {make_float2(h4.x, h4.y), make_float2(h4.z, h4.w)}, acc = f2(0.f);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const float2 e = ex2_pair(__fmul2_rn(f2(di), c.A2[p]));
                h[p] = __ffma2_rn(e, h[p], input_term<ZOH>(f2(di), f2(xi), e, c.A2[p], c.Ar[p], bq[p]));
                acc = __ffma2_rn(cq[p], h[p], acc);
                finite = __ffma2_rn(h[p], f2(0.f), finite);
            }
            yp[i] = acc.x + acc.y;
            if (dv) *reinterpret_cast<float4*>(row_at(pool, k, entry)) = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
        }
        real::reduce_scatter<R, NG>(yp, ng);
#pragma unroll
        for (int j = 0; j < SH; ++j) {
            float v = fmaf(c.dsk, x[j], yp[j]);
            if (pz) v *= silu_fast(z[j]);
            if (dv && ky[j] >= 0) *row_at(py, r + ng * SH + j, ldy) = Elem<E>::from_f(v);
        }
        stage = stage == kStepStages - 1 ? 0 : stage + 1;
    }
    if (dv && !(finite.x + finite.y == 0.f)) flag_if(a.status, kStatusNonFinite);
}

template <typename E, int N, bool ZOH, bool MANY>
cudaError_t prompt_launch(const ScanServeArgs& a, unsigned ctas, cudaStream_t st) {
    scan_prompt_kernel<E, N, ZOH, MANY><<<ctas, PromptCfg<N, MANY>::NW * 32, 0, st>>>(a);
    return cudaGetLastError();
}

// The forms cross where the few form's throughput meets the time that the longest sequence takes in the many
// form, that is at a fixed number of CTAs' worth of full-length work, rows * ndt / max_len.  Measured on a
// B200 (bf16, gated; us many / few): N = 16 at 351 201 / 166, at 411 56 / 84, at 678 48 / 76; N = 8 at 245
// 158 / 108, at 339 34 / 43; N = 4 at 192 41 / 34, at 429 16 / 34.  Without the caller's max_len it is the rows, as
// of one sequence, and the few form is taken below kManyFrom tiles: 24 prompts of 9989 rows on 4096 channels then
// take 481 us instead of 326.
template <int N> constexpr int64_t kManyFrom = N == 16 ? 363 : (N == 8 ? 300 : 250);

template <typename E, int N, bool ZOH>
cudaError_t prompt_impl(ScanServeArgs a, cudaStream_t st) {
    a.ndt = (a.D + PromptCfg<N, true>::CW - 1) / PromptCfg<N, true>::CW;
    const int64_t ctas = (int64_t)a.S * a.ndt;
    // Worth it when there are more CTAs than run at once, few enough sequences to be ranked by every CTA, and
    // a longest one (36 cycles a step) that outweighs the ranking, 2 us a CTA.
    a.sorted = a.S > 1 && a.S <= 64 && ctas > 592 && a.max_len >= 512 &&
               (int64_t)a.max_len * a.S > 2 * (int64_t)a.rows;
    if ((int64_t)a.rows * a.ndt >= kManyFrom<N> * a.max_len)
        return prompt_launch<E, N, ZOH, true>(a, (unsigned)ctas, st);
    return prompt_launch<E, N, ZOH, false>(a, (unsigned)ctas, st);
}

template <typename E, int N>
cudaError_t prompt_pick(const ScanServeArgs& a, cudaStream_t st) {
    return a.zoh ? prompt_impl<E, N, true>(a, st) : prompt_impl<E, N, false>(a, st);
}

template <typename E>
cudaError_t prompt_dispatch(const ScanServeArgs& a, int N, cudaStream_t st) {
    if (N == 4) return prompt_pick<E, 4>(a, st);
    if (N == 8) return prompt_pick<E, 8>(a, st);
    return prompt_pick<E, 16>(a, st);
}

// One row a CTA while those CTAs run at once (8 an SM); else as many rows a CTA as leave one wave of three
// CTAs an SM, in whole groups, at most kStepRows.
template <typename E, int N, bool ZOH>
cudaError_t step_impl(const ScanServeArgs& a, cudaStream_t st) {
    constexpr int DC = 256 / (N / 4);
    const int64_t tiles = (a.D + DC - 1) / DC;
    if (tiles * a.rows <= 1184) {
        scan_step_kernel<E, N, ZOH><<<dim3((unsigned)tiles, a.rows), 256, 0, st>>>(a);
    } else {
        const int64_t groups = tiles < 444 ? 444 / tiles : 1;
        int64_t rows = ((a.rows + groups - 1) / groups + kStepGroup - 1) / kStepGroup * kStepGroup;
        if (rows > kStepRows) rows = kStepRows;
        const int smem = StepCfg<N>::kBytes;
        const cudaError_t e = cudaFuncSetAttribute(scan_step_batch_kernel<E, N, ZOH>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        scan_step_batch_kernel<E, N, ZOH>
            <<<dim3((unsigned)tiles, (unsigned)((a.rows + rows - 1) / rows)), 256, smem, st>>>(a, (int)rows);
    }
    return cudaGetLastError();
}

template <typename E, int N>
cudaError_t step_pick(const ScanServeArgs& a, cudaStream_t st) {
    return a.zoh ? step_impl<E, N, true>(a, st) : step_impl<E, N, false>(a, st);
}

template <typename E>
cudaError_t step_dispatch(const ScanServeArgs& a, int N, cudaStream_t st) {
    if (N == 4) return step_pick<E, 4>(a, st);
    if (N == 8) return step_pick<E, 8>(a, st);
    return step_pick<E, 16>(a, st);
}

}  // namespace
}  // namespace serve

cudaError_t launch_scan_prompt(const ScanServeArgs& a, int io_bf16, int N, cudaStream_t st) {
    return io_bf16 ? serve::prompt_dispatch<__nv_bfloat16>(a, N, st)
                   : serve::prompt_dispatch<float>(a, N, st);
}

cudaError_t launch_scan_step(const ScanServeArgs& a, int io_bf16, int N, cudaStream_t st) {
    return io_bf16 ? serve::step_dispatch<__nv_bfloat16>(a, N, st) : serve::step_dispatch<float>(a, N, st);
}

}  // namespace ssm
