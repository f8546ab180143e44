// Selective scan for serving: packed prompts of different lengths, and single tokens, on a pool of
// states (include/ssm_scan.h).
//
//     h_t = exp(delta_t A) h_{t-1} + w_t B_t x_t,   y_t = (C_t . h_t + D x_t) [z_t sigmoid(z_t)],
//     w = delta (Euler) or (exp(delta A) - 1) / A (zero-order hold).
//
// Prompts.  What bounds a long prompt is the exp2 unit: one exp2 a state and step (16 lanes a
// cycle and SM, so 8 cycles a warp instruction) against 4 packed fp32 instructions for two states;
// memory traffic is 8 bytes a channel and step in bf16, a small share.  So nothing may stand between
// the exp2s: a warp needs no other warp except for B and C, which a CTA converts to fp32 in shared
// memory once for its channels, double-buffered, one barrier per 32 steps.  A channel's N states
// are spread over NG adjacent lanes; a lane reads x, delta and z of its share of eight steps straight
// from global memory (one group ahead), evaluates their softplus and gate once, hands (delta,
// delta x) to its neighbours by shuffles, and the reduce-scatter of the eight y's over the lanes
// leaves each lane the y's of the same steps, so y is gated and stored by the lane that holds z.
// With NG = 1 (all states in one thread) there are no shuffles and the fewest instructions a state;
// with NG = N / 4 a batch has four times the threads.
//
// Time split.  A sequence longer than G rows runs as segments: a first launch scans every segment
// but the last from zero (end state and transition product), the carry turns these into the
// states entering the segments, and the scan runs from them.  That evaluates every exp2 of a
// split sequence twice, so it is done only when the unsplit batch would leave the GPU waiting for
// its longest sequence (plan_scan_prompt).
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
// channels a CTA.  Each of its warps holds all of them, for its turns of U steps.  Row by row a lane
// holds SH of the turn's steps, the same ones whose sums the reduction over the NG lanes leaves in it.
template <int N>
struct PromptCfg {
    static constexpr int NG = N / 4;
    static constexpr int CW = 64 / NG;
    static constexpr int U = N == 4 ? 4 : 8;
    static constexpr int SH = U / NG;
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

template <typename E, int N, bool ZOH, int NW>
__global__ void __launch_bounds__(NW * 32, 12 / NW) scan_prompt_kernel(ScanServeArgs a) {
    using Cfg = PromptCfg<N>;
    using PR = typename Pair<E>::Raw;
    using BR = typename Vec<E, 4>::Raw;
    constexpr int NG = Cfg::NG, CW = Cfg::CW, U = Cfg::U, SH = Cfg::SH, NP = CW / 2;
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
        A2[c][0] = make_float2(-expf(l[c].x) * kLog2e, -expf(l[c].y) * kLog2e);
        A2[c][1] = make_float2(-expf(l[c].z) * kLog2e, -expf(l[c].w) * kLog2e);
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
        // the transitions: nothing here waits for the state
        float2 e[U][2][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float2 dlt = s_dlt[warp][u][dl];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                e[u][0][p] = ex2_pair(__fmul2_rn(f2(dlt.x), A2[0][p]));
                e[u][1][p] = ex2_pair(__fmul2_rn(f2(dlt.y), A2[1][p]));
            }
        }
        // the recurrence, from the warp before to the warp after; e[u] becomes the state at step u
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
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float2 bq[2];
            Vec<E, 4>::unpack(s_b[warp][u * NG + ng], bq);
            const float2 dx = s_dx[warp][u][dl];
            float2 dlt = f2(0.f);
            if (ZOH) dlt = s_dlt[warp][u][dl];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const float2 w0 = input_term<ZOH>(f2(dlt.x), f2(dx.x), e[u][0][p], A2[0][p], Ar[0][p], bq[p]);
                const float2 w1 = input_term<ZOH>(f2(dlt.y), f2(dx.y), e[u][1][p], A2[1][p], Ar[1][p], bq[p]);
                h[0][p] = e[u][0][p] = __ffma2_rn(e[u][0][p], h[0][p], w0);
                h[1][p] = e[u][1][p] = __ffma2_rn(e[u][1][p], h[1][p], w1);
            }
        }
        if (i + 1 < turns) {
            const int to = warp + 1 == NW ? 0 : warp + 1;
#pragma unroll
            for (int c = 0; c < 2; ++c) s_h[to][c][lane] = make_float4(h[c][0].x, h[c][0].y, h[c][1].x, h[c][1].y);
            hand_over(to);
        } else {
            if (entry)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    *reinterpret_cast<float4*>(entry + c * N) = make_float4(h[c][0].x, h[c][0].y, h[c][1].x, h[c][1].y);
            if (dv && !(real::all_finite<4>(h[0]) && real::all_finite<4>(h[1]))) flag_if(a.status, kStatusNonFinite);
        }
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
// Four states a thread, N / 4 lanes a channel, R rows a CTA: the transition's A is computed once
// for the R rows and their states are in flight together.  Lane ng of a channel evaluates the softplus
// and the gate of row ng (R <= N / 4 lanes) and hands them to its neighbours.
template <typename E, int N, int R, bool ZOH>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanServeArgs a) {
    constexpr int NG = N / 4, DC = 256 / NG;
    const int tid = threadIdx.x, ng = tid % NG, dl = tid / NG, n0 = ng * 4;
    const int d = blockIdx.x * DC + dl;
    const bool dv = d < a.D;
    const int row0 = blockIdx.y * R;

    int k[R];
    float4 h4[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = row0 + r;
        k[r] = row < a.rows ? (a.slot ? a.slot[row] : row) : -1;
        const bool work = dv && k[r] >= 0 && k[r] < a.slots;
        h4[r] = work ? *reinterpret_cast<const float4*>(a.pool + ((size_t)k[r] * a.D + d) * N + n0)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    typename Vec<E, 4>::Raw rB[R], rC[R];
    E x[R], dr[R], z[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool work = dv && k[r] >= 0 && k[r] < a.slots;
        const size_t row = work ? row0 + r : 0;
        rB[r] = work ? ld_vec<E, 4>(static_cast<const E*>(a.Bm) + row * a.ldb + n0) : Vec<E, 4>::zero();
        rC[r] = work ? ld_vec<E, 4>(static_cast<const E*>(a.Cm) + row * a.ldc + n0) : Vec<E, 4>::zero();
        x[r] = work ? static_cast<const E*>(a.x)[row * a.ldx + d] : Elem<E>::from_f(0.f);
        dr[r] = work ? static_cast<const E*>(a.draw)[row * a.ldd + d] : Elem<E>::from_f(0.f);
        z[r] = work && a.z ? static_cast<const E*>(a.z)[row * a.ldz + d] : Elem<E>::from_f(0.f);
    }
    const float4 l = dv ? __ldg(reinterpret_cast<const float4*>(a.A_log + (size_t)d * N + n0))
                        : make_float4(0.f, 0.f, 0.f, 0.f);
    const float dsk = dv ? a.Dskip[d] : 0.f;
    if (a.slot) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = k[r] >= 0 && k[r] < a.slots;
            const bool rep = __syncthreads_or(named_before(a.slot, row0 + r, in ? k[r] : -1, tid, 256));
            if (rep || k[r] >= a.slots) {
                if (tid == 0 && blockIdx.x == 0) flag_if(a.status, kStatusInvalid);
                k[r] = -1;
            }
        }
    }
    const float2 A2[2] = {make_float2(-expf(l.x) * kLog2e, -expf(l.y) * kLog2e),
                          make_float2(-expf(l.z) * kLog2e, -expf(l.w) * kLog2e)};
    float2 Ar[2];
    if (ZOH) {
        Ar[0] = make_float2(-expf(-l.x), -expf(-l.y));
        Ar[1] = make_float2(-expf(-l.z), -expf(-l.w));
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float xf = Elem<E>::to_f(x[r]);
        const float dlt = softplus_fast(Elem<E>::to_f(dr[r]));
        const float2 dd = make_float2(dlt, dlt * xf);
        float2 bq[2], cq[2], acc = f2(0.f);
        Vec<E, 4>::unpack(rB[r], bq);
        Vec<E, 4>::unpack(rC[r], cq);
        float2 h[2] = {make_float2(h4[r].x, h4[r].y), make_float2(h4[r].z, h4[r].w)};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 zl2 = __fmul2_rn(f2(dd.x), A2[i]);
            const float2 e = ex2_pair(zl2);
            h[i] = __ffma2_rn(e, h[i], input_term<ZOH>(f2(dd.x), f2(dd.y), e, A2[i], Ar[i], bq[i]));
            acc = __ffma2_rn(cq[i], h[i], acc);
        }
        float v = acc.x + acc.y;
#pragma unroll
        for (int m = 1; m < NG; m <<= 1) v += __shfl_xor_sync(kFull, v, m);
        if (!dv || k[r] < 0) continue;
        *reinterpret_cast<float4*>(a.pool + ((size_t)k[r] * a.D + d) * N + n0) =
            make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
        if (!real::all_finite<4>(h)) flag_if(a.status, kStatusNonFinite);
        if (ng == 0) {
            v = fmaf(dsk, xf, v);
            if (a.z) v *= silu_fast(Elem<E>::to_f(z[r]));
            static_cast<E*>(a.y)[(size_t)(row0 + r) * a.ldy + d] = Elem<E>::from_f(v);
        }
    }
}

template <typename E, int N, bool ZOH>
cudaError_t prompt_impl(ScanServeArgs a, cudaStream_t st) {
    constexpr int CW = PromptCfg<N>::CW;
    a.ndt = (a.D + CW - 1) / CW;
    const int64_t ctas = (int64_t)a.S * a.ndt;
    // worth it when there are more CTAs than run at once, and few enough sequences to be ranked by every CTA
    a.sorted = a.S > 1 && a.S <= 64 && ctas > 296 && (int64_t)a.max_len * a.S > 2 * (int64_t)a.rows;
    if (ctas <= 148)
        scan_prompt_kernel<E, N, ZOH, 12><<<(unsigned)ctas, 12 * 32, 0, st>>>(a);
    else
        scan_prompt_kernel<E, N, ZOH, 6><<<(unsigned)ctas, 6 * 32, 0, st>>>(a);
    return cudaGetLastError();
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

template <typename E, int N, int R>
cudaError_t step_impl(const ScanServeArgs& a, cudaStream_t st) {
    constexpr int DC = 256 / (N / 4);
    const dim3 grid((a.D + DC - 1) / DC, (a.rows + R - 1) / R);
    if (a.zoh)
        scan_step_kernel<E, N, R, true><<<grid, 256, 0, st>>>(a);
    else
        scan_step_kernel<E, N, R, false><<<grid, 256, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename E, int N>
cudaError_t step_pick(const ScanServeArgs& a, cudaStream_t st) {
    // four rows a CTA once one row a CTA gives more CTAs than are resident (8 per SM)
    constexpr int DC = 256 / (N / 4);
    if ((int64_t)((a.D + DC - 1) / DC) * a.rows > 1184) return step_impl<E, N, 4>(a, st);
    return step_impl<E, N, 1>(a, st);
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
