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

constexpr int kTT = 32;   // steps per staged tile of B and C
constexpr int kU = 8;     // steps per unrolled group
constexpr int kThreads = 128;

// four B or C elements of a row, as fp32
template <typename E>
__device__ __forceinline__ float4 quad_f4(const typename Vec<E, 4>::Raw& r) {
    float2 o[2];
    Vec<E, 4>::unpack(r, o);
    return make_float4(o[0].x, o[0].y, o[1].x, o[1].y);
}

// w B x for a pair of states: (delta, delta x), a = exp(delta A), zl2 = delta A log2(e), Ar = 1 / A
template <bool ZOH>
__device__ __forceinline__ float2 input_term(float2 dd, float2 a, float2 zl2, float2 Ar, float2 bq) {
    if constexpr (ZOH) {
        const float2 z = __fmul2_rn(zl2, f2(kLn2));
        const float2 rz = __fmul2_rn(f2(__fdividef(1.0f, dd.x)), Ar);
        return __fmul2_rn(__fmul2_rn(f2(dd.y), real::zoh_e1(z, a, rz)), bq);
    } else {
        return __fmul2_rn(f2(dd.y), bq);
    }
}

// S states from S/4 16-byte vectors
template <int S>
__device__ __forceinline__ void ld_state(float2 (&h)[S / 2], const float* p) {
    real::ld_pairs<S>(h, p);
}

template <typename E, int N, int S, bool ZOH, bool SUMMARY>
__global__ void __launch_bounds__(kThreads) scan_prompt_kernel(ScanServeArgs a) {
    constexpr int NG = N / S, DC = kThreads / NG, P2 = S / 2, SH = kU / NG;  // SH: steps of a lane's share
    constexpr int NQ = kTT * N / 4;                                  // four-element vectors of a B tile
    constexpr int PER = (NQ + kThreads - 1) / kThreads;
    __shared__ __align__(16) float sB[2][kTT * N];
    __shared__ __align__(16) float sC[SUMMARY ? 1 : 2][SUMMARY ? 4 : kTT * N];
    const int64_t item = blockIdx.x / a.ndt;
    const int tile = blockIdx.x % a.ndt;
    const int tid = threadIdx.x, ng = tid % NG, dl = tid / NG;
    const int d = tile * DC + dl, n0 = ng * S;
    const bool dv = d < a.D;

    if (!SUMMARY && a.status && blockIdx.x == 0)
        check_batch(a.offsets, a.slot, a.S, a.rows, a.slots, a.max_len, a.status);
    const int s = find_seq(a.offsets, a.S, a.G, item);
    const Span sp = item_span(a.offsets, a.slot, s, a.G, item, a.rows, a.slots, a.max_len);
    if (!sp.ok) return;  // the whole CTA
    const int n = min(a.G, sp.end - sp.first);  // this segment's steps
    const bool last = sp.first + n == sp.end;
    if (SUMMARY && last) return;
    if (__syncthreads_or(named_before(a.slot, s, sp.slot, tid, kThreads))) {
        if (!SUMMARY && tid == 0) flag_if(a.status, kStatusInvalid);
        return;
    }

    float2 A2[P2], Ar[P2], h[P2];
#pragma unroll
    for (int i = 0; i < P2; ++i) {
        const float l0 = dv ? a.A_log[(size_t)d * N + n0 + 2 * i] : 0.f;
        const float l1 = dv ? a.A_log[(size_t)d * N + n0 + 2 * i + 1] : 0.f;
        A2[i] = make_float2(-expf(l0) * kLog2e, -expf(l1) * kLog2e);
        if (ZOH) Ar[i] = make_float2(-expf(-l0), -expf(-l1));
        h[i] = f2(0.f);
    }
    float* entry = sp.slot >= 0 ? a.pool + ((size_t)sp.slot * a.D + d) * N + n0 : nullptr;
    if (!SUMMARY && dv) {
        if (sp.local > 0)  // the carry's state entering this segment
            ld_state<S>(h, a.sumS + ((size_t)item * a.D + d) * N + n0);
        else if (entry && a.carry && a.carry[s])
            ld_state<S>(h, entry);
    }
    const float dsk = !SUMMARY && dv ? a.Dskip[d] : 0.f;
    float dsum = 0.f;  // summary: sum of delta over the lane's own steps

    const size_t r0 = (size_t)sp.first;
    const E* px = static_cast<const E*>(a.x) + r0 * a.ldx + (dv ? d : 0);
    const E* pd = static_cast<const E*>(a.draw) + r0 * a.ldd + (dv ? d : 0);
    const E* pz = !SUMMARY && a.z ? static_cast<const E*>(a.z) + r0 * a.ldz + (dv ? d : 0) : nullptr;
    E* py = SUMMARY ? nullptr : static_cast<E*>(a.y) + r0 * a.ldy + d;
    const E* pB = static_cast<const E*>(a.Bm) + r0 * a.ldb;
    const E* pC = static_cast<const E*>(a.Cm) + r0 * a.ldc;

    // B and C of steps [t, t + 32): zero past the segment's end, so that a step which is not there
    // (delta = 0: transition one) adds nothing to the state
    typename Vec<E, 4>::Raw rB[PER], rC[PER];
    auto fetch = [&](int t) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int q = tid + i * kThreads, row = q / (N / 4), col = (q % (N / 4)) * 4;
            const bool ok = q < NQ && t + row < n;
            rB[i] = ok ? ld_vec<E, 4>(pB + (size_t)(t + row) * a.ldb + col) : Vec<E, 4>::zero();
            if (!SUMMARY) rC[i] = ok ? ld_vec<E, 4>(pC + (size_t)(t + row) * a.ldc + col) : Vec<E, 4>::zero();
        }
    };
    auto stage = [&](int k) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int q = tid + i * kThreads;
            if (q < NQ) {
                reinterpret_cast<float4*>(sB[k])[q] = quad_f4<E>(rB[i]);
                if (!SUMMARY) reinterpret_cast<float4*>(sC[SUMMARY ? 0 : k])[q] = quad_f4<E>(rC[i]);
            }
        }
    };
    // the lane's share of the group at t: steps t + ng * SH + j
    E nx[SH], nd[SH], nz[SH];
    auto next = [&](int t) {
#pragma unroll
        for (int j = 0; j < SH; ++j) {
            const int r = t + ng * SH + j;
            const bool ok = r < n;
            nx[j] = ok ? px[(size_t)r * a.ldx] : Elem<E>::from_f(0.f);
            nd[j] = ok ? pd[(size_t)r * a.ldd] : Elem<E>::from_f(0.f);
            if (!SUMMARY) nz[j] = ok && pz ? pz[(size_t)r * a.ldz] : Elem<E>::from_f(0.f);
        }
    };

    fetch(0);
    next(0);
    for (int t0 = 0, k = 0; t0 < n; t0 += kTT, k ^= 1) {
        stage(k);
        __syncthreads();  // also: everyone has left the tile before last, whose buffer is next
        if (t0 + kTT < n) fetch(t0 + kTT);
        const int tend = min(n, t0 + kTT);
        for (int t = t0; t < tend; t += kU) {
            float dlt[SH], dx[SH], xs[SH], zs[SH];
#pragma unroll
            for (int j = 0; j < SH; ++j) {
                const bool ok = t + ng * SH + j < n;
                xs[j] = Elem<E>::to_f(nx[j]);
                zs[j] = SUMMARY ? 0.f : Elem<E>::to_f(nz[j]);
                dlt[j] = ok ? softplus_fast(Elem<E>::to_f(nd[j])) : 0.f;
                dx[j] = dlt[j] * xs[j];
                if (SUMMARY) dsum += dlt[j];
            }
            next(t + kU);
            float yp[kU];
            const float* tB = sB[k] + (t - t0) * N + n0;
            const float* tC = sC[SUMMARY ? 0 : k] + (SUMMARY ? 0 : (t - t0) * N + n0);
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                float2 dd = make_float2(dlt[u % SH], dx[u % SH]);
                if (NG > 1) {
                    dd.x = __shfl_sync(kFull, dd.x, u / SH, NG);
                    dd.y = __shfl_sync(kFull, dd.y, u / SH, NG);
                }
                float2 bq[P2], cq[P2], acc = f2(0.f);
                real::ld_pairs<S>(bq, tB + u * N);
                if (!SUMMARY) real::ld_pairs<S>(cq, tC + u * N);
#pragma unroll
                for (int i = 0; i < P2; ++i) {
                    const float2 zl2 = __fmul2_rn(f2(dd.x), A2[i]);
                    const float2 e = ex2_pair(zl2);
                    h[i] = __ffma2_rn(e, h[i], input_term<ZOH>(dd, e, zl2, Ar[i], bq[i]));
                    if (!SUMMARY) acc = __ffma2_rn(cq[i], h[i], acc);
                }
                yp[u] = acc.x + acc.y;
            }
            if (!SUMMARY) {
                real::reduce_scatter<kU, NG>(yp, ng);
#pragma unroll
                for (int j = 0; j < SH; ++j) {
                    const int r = t + ng * SH + j;
                    float v = fmaf(dsk, xs[j], yp[j]);
                    if (pz) v *= silu_fast(zs[j]);
                    if (dv && r < n) py[(size_t)r * a.ldy] = Elem<E>::from_f(v);
                }
            }
        }
    }
    if (SUMMARY) {
        // the product of the transitions is exp(A sum delta): the lanes' sums, added over the channel
#pragma unroll
        for (int m = 1; m < NG; m <<= 1) dsum += __shfl_xor_sync(kFull, dsum, m);
        if (dv) {
            float2 P[P2];
#pragma unroll
            for (int i = 0; i < P2; ++i) P[i] = ex2_pair(__fmul2_rn(f2(dsum), A2[i]));
            const size_t o = ((size_t)item * a.D + d) * N + n0;
            real::st_pairs<S>(a.sumP + o, P);
            real::st_pairs<S>(a.sumS + o, h);
        }
    } else if (dv && last) {
        if (entry) real::st_pairs<S>(entry, h);
        if (!real::all_finite<S>(h)) flag_if(a.status, kStatusNonFinite);
    }
}

// The states entering the segments of each sequence, written over the segments' end states (segment
// i's entering state in place of segment i's own sum): four states a thread.
__global__ void __launch_bounds__(256) scan_carry_kernel(ScanServeArgs a, int DN4) {
    const int s = blockIdx.y, k = blockIdx.x * 256 + threadIdx.x;
    const int64_t base = item_base(a.offsets, s, a.G);
    const Span sp = item_span(a.offsets, a.slot, s, a.G, base, a.rows, a.slots, a.max_len);
    const int len = sp.ok ? sp.end - sp.first : 0;
    const int nseg = (len + a.G - 1) / a.G;
    if (nseg < 2) return;  // the whole CTA: nothing to carry
    if (__syncthreads_or(named_before(a.slot, s, sp.slot, threadIdx.x, 256))) return;
    if (k >= DN4) return;
    float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
    if (sp.slot >= 0 && a.carry && a.carry[s])
        h = reinterpret_cast<const float4*>(a.pool)[(size_t)sp.slot * DN4 + k];
    const float4* P = reinterpret_cast<const float4*>(a.sumP) + (size_t)base * DN4 + k;
    float4* E = reinterpret_cast<float4*>(a.sumS) + (size_t)base * DN4 + k;
#pragma unroll 4
    for (int i = 0; i < nseg; ++i) {
        float4 p, e;
        if (i + 1 < nseg) { p = P[(size_t)i * DN4]; e = E[(size_t)i * DN4]; }
        E[(size_t)i * DN4] = h;
        if (i + 1 < nseg)
            h = make_float4(fmaf(p.x, h.x, e.x), fmaf(p.y, h.y, e.y), fmaf(p.z, h.z, e.z), fmaf(p.w, h.w, e.w));
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
            h[i] = __ffma2_rn(e, h[i], input_term<ZOH>(dd, e, zl2, Ar[i], bq[i]));
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

template <typename E, int N, int S, bool ZOH>
cudaError_t prompt_impl(ScanServeArgs a, cudaStream_t st) {
    constexpr int DC = kThreads / (N / S);
    a.ndt = (a.D + DC - 1) / DC;
    const unsigned grid = (unsigned)(a.items * a.ndt);
    cudaError_t e;
    if (a.split) {
        scan_prompt_kernel<E, N, S, ZOH, true><<<grid, kThreads, 0, st>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        const int DN4 = a.D * (N / 4);
        scan_carry_kernel<<<dim3((DN4 + 255) / 256, a.S), 256, 0, st>>>(a, DN4);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    scan_prompt_kernel<E, N, S, ZOH, false><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename E, int N>
cudaError_t prompt_pick(const ScanServeArgs& a, int states, cudaStream_t st) {
    if (states == N) return a.zoh ? prompt_impl<E, N, N, true>(a, st) : prompt_impl<E, N, N, false>(a, st);
    return a.zoh ? prompt_impl<E, N, 4, true>(a, st) : prompt_impl<E, N, 4, false>(a, st);
}

template <typename E>
cudaError_t prompt_dispatch(const ScanServeArgs& a, int N, int states, cudaStream_t st) {
    if (N == 4) return prompt_pick<E, 4>(a, states, st);
    if (N == 8) return prompt_pick<E, 8>(a, states, st);
    return prompt_pick<E, 16>(a, states, st);
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

ScanServePlan plan_scan_prompt(int64_t rows, int64_t S, int64_t D, int N, int64_t max_len) {
    ScanServePlan p;
    p.states = 4;
    const int64_t dc = serve::kThreads / (N / p.states), ndt = (D + dc - 1) / dc;
    // steps of one of 1184 CTAs (8 per SM) if the batch were spread evenly
    const int64_t even = rows * ndt / 1184;
    int64_t G = max_len;
    if (max_len > 2 * even && max_len > 128) G = (even > 64 ? even : 64);
    G = (G + 31) / 32 * 32;
    if (G < 32) G = 32;
    p.G = (int)G;
    p.split = max_len > G;
    p.items = rows / G + S;
    return p;
}

cudaError_t launch_scan_prompt(const ScanServeArgs& a, int io_bf16, int N, int states, cudaStream_t st) {
    return io_bf16 ? serve::prompt_dispatch<__nv_bfloat16>(a, N, states, st)
                   : serve::prompt_dispatch<float>(a, N, states, st);
}

cudaError_t launch_scan_step(const ScanServeArgs& a, int io_bf16, int N, cudaStream_t st) {
    return io_bf16 ? serve::step_dispatch<__nv_bfloat16>(a, N, st) : serve::step_dispatch<float>(a, N, st);
}

}  // namespace ssm
