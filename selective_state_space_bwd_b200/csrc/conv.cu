// Short causal convolution in front of the scan: forward, its recomputation from an 8-bit
// checkpoint, its gradient, and the packed-prompt and single-token forms (include/ssm_scan.h).
//
// Every kernel is bound by memory traffic: 2 W + ~8 operations an element against 4 (forward, bf16)
// to 6 bytes (backward).  A thread owns four consecutive channels (one fp32x2 pair each of two) and
// walks down a piece of the rows, the last W-1 inputs in registers, so that an element is read once
// from DRAM; the W-1 rows before a piece are read a second time (from L2).  Four channels, not
// eight: the gradient keeps W taps, W+1 sums and two windows a channel, and at four channels two
// CTAs of 256 threads stay resident.  A CTA is cx threads across (cx four-channel vectors, a multiple of
// eight so that the eight lanes that share an 8-bit group's 32 channels are neighbours in a warp)
// by ry pieces down; cx is D / 4 cut into equal column tiles of at most 32, so that a width just
// past a tile leaves no tile empty.
#include "layer_common.cuh"

namespace ssm {
namespace conv {
namespace {

constexpr int U = 4;  // rows whose loads are in flight ahead of the rows being computed

// cx multiples of 8 up to 32, ry = 256 / cx
struct Tile {
    int cx, ry, nct;
};
Tile tile_of(int D) {
    const int nvec = (D + 31) / 32 * 8;
    Tile t;
    t.nct = (nvec + 31) / 32;
    t.cx = ((nvec + t.nct - 1) / t.nct + 7) / 8 * 8;
    t.ry = 256 / t.cx;
    return t;
}

// The taps of four channels, tap-major: w[j][pair].
template <int W>
__device__ __forceinline__ void load_taps(float2 (&w)[W][2], float2 (&bias)[2], const float* pw,
                                          const float* pb, int c) {
    float f[4 * W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(pw + (size_t)c * W) + i);
        f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
    }
#pragma unroll
    for (int j = 0; j < W; ++j) {
        w[j][0] = make_float2(f[j], f[W + j]);
        w[j][1] = make_float2(f[2 * W + j], f[3 * W + j]);
    }
    const float4 b = pb ? __ldg(reinterpret_cast<const float4*>(pb + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
    bias[0] = make_float2(b.x, b.y);
    bias[1] = make_float2(b.z, b.w);
}

template <int W>
__device__ __forceinline__ void preact(float2 (&v)[2], const float2 (&w)[W][2],
                                       const float2 (&bias)[2], const float2 (*x)[2]) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        v[p] = bias[p];
#pragma unroll
        for (int j = 0; j < W; ++j) v[p] = __ffma2_rn(w[j][p], x[j][p], v[p]);
    }
}

__device__ __forceinline__ void silu4(float2 (&v)[2]) {
#pragma unroll
    for (int p = 0; p < 2; ++p) v[p] = make_float2(silu_fast(v[p].x), silu_fast(v[p].y));
}

// ---------------------------------------------------------------- 8-bit checkpoint
// The step of magnitudes from 2^127 on: 64 of twice that would be 2^128, so there 127 steps are
// the limit instead.
constexpr unsigned kTopStep = 248u;

// The biased exponent of a group's step from the largest magnitude's bits (an unsigned maximum, so
// that a NaN, above every number's bits, is not lost as fmaxf would lose it).
__device__ __forceinline__ unsigned step_exponent(unsigned top) {
    if (top == 0u) return 0u;
    const unsigned e = top >> 23;
    if (e == 255u) return 255u;
    unsigned q = e > 7u ? e - 6u : 1u;
    // 2^-(step): q is at most kTopStep, so the factor is a normal number
    if (q < kTopStep && __uint_as_float(top) * __uint_as_float((254u - q) << 23) >= 127.5f) ++q;
    return q;
}

// Four int8 of x / 2^(qe - 127), rounded to nearest even: adding 1.5 * 2^23 leaves the rounded
// integer in the low bits of the sum (the product by a power of two is exact).
__device__ __forceinline__ unsigned quantise4(float2 (&x)[2], unsigned qe) {
    if (qe == 0u || qe == 255u) return 0u;
    const float f = __uint_as_float((254u - qe) << 23);
    if (qe == kTopStep) {
        const float m = 127.0f * __uint_as_float(kTopStep << 23);
#pragma unroll
        for (int p = 0; p < 2; ++p)
            x[p] = make_float2(fminf(fmaxf(x[p].x, -m), m), fminf(fmaxf(x[p].y, -m), m));
    }
    const float magic = 12582912.0f;
    const float2 a = __ffma2_rn(x[0], make_float2(f, f), make_float2(magic, magic));
    const float2 b = __ffma2_rn(x[1], make_float2(f, f), make_float2(magic, magic));
    const unsigned lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
    const unsigned hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}

// The values of four int8.  A byte u = q + 128 in the low bits of 2^23 is the float 2^23 + u; the
// step of a NaN group (exponent 255) is infinite and its q zero, and 0 * inf is the NaN wanted.
__device__ __forceinline__ void restore4(float2 (&x)[2], unsigned q, unsigned qe) {
    const float step = __uint_as_float(qe << 23);
    const unsigned u = q ^ 0x80808080u;
    const float off = -8388736.0f;  // -(2^23 + 128)
    const float2 o = make_float2(off, off), s = make_float2(step, step);
    const float2 a = make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540)),
                                 __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7541)));
    const float2 b = make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7542)),
                                 __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7543)));
    x[0] = __fmul2_rn(__fadd2_rn(a, o), s);
    x[1] = __fmul2_rn(__fadd2_rn(b, o), s);
}

// ---------------------------------------------------------------- row sources
// One row's four channels of one batch entry, from x or from its 8-bit checkpoint.
template <typename E, bool Q8> struct Rows;
template <typename E> struct Rows<E, false> {
    using Raw = typename Quad<E>::Raw;
    const E* x;
    size_t ld;
    __device__ __forceinline__ Rows(const ConvArgs& a, int b, int c)
        : x(static_cast<const E*>(a.x) + (size_t)b * a.L * a.ldx + c), ld(a.ldx) {}
    __device__ __forceinline__ Raw load(int t) const { return ld_quad(x + (size_t)t * ld); }
    static __device__ __forceinline__ Raw zero() { return Quad<E>::zero(); }
    static __device__ __forceinline__ void unpack(const Raw& r, float2 (&o)[2]) { Quad<E>::unpack(r, o); }
};
template <typename E> struct Rows<E, true> {
    struct Raw { unsigned q, e; };
    const int8_t* q;
    const uint8_t* e;
    size_t D, ng;
    __device__ __forceinline__ Rows(const ConvArgs& a, int b, int c)
        : q(a.q + (size_t)b * a.L * a.D + c), e(a.qe + (size_t)b * a.L * ((a.D + 31) / 32) + c / 32),
          D(a.D), ng((a.D + 31) / 32) {}
    __device__ __forceinline__ Raw load(int t) const {
        return Raw{*reinterpret_cast<const unsigned*>(q + (size_t)t * D), e[(size_t)t * ng]};
    }
    static __device__ __forceinline__ Raw zero() { return Raw{0u, 0u}; }
    static __device__ __forceinline__ void unpack(const Raw& r, float2 (&o)[2]) { restore4(o, r.q, r.e); }
};

// Row t < 0 of a sequence: the state before it, or zero.
template <typename E, int W>
__device__ __forceinline__ void past_row(float2 (&o)[2], const E* s0, int t, size_t D) {
    if (s0)
        Quad<E>::unpack(ld_quad(s0 + (size_t)(t + W - 1) * D), o);
    else
        o[0] = o[1] = make_float2(0.f, 0.f);
}

// ---------------------------------------------------------------- forward
// SRC8: from the checkpoint (restore); DST8: write the checkpoint.
template <typename E, int W, bool SILU, bool SRC8, bool DST8>
__global__ void __launch_bounds__(256) conv_fwd_kernel(ConvArgs a) {
    const int tx = threadIdx.x % a.cx, ty = threadIdx.x / a.cx;
    const int64_t piece = (int64_t)blockIdx.x * a.ry + ty;
    if (piece >= (int64_t)a.B * a.nseg) return;  // whole rows of threads: whole groups of eight lanes
    const int c = (blockIdx.y * a.cx + tx) * 4;
    const bool cv = c < a.D;
    const int b = (int)(piece / a.nseg), seg = (int)(piece % a.nseg);
    const int t0 = seg * a.G, t1 = min(a.L, t0 + a.G);
    if (!DST8 && !cv) return;
    const int cc = cv ? c : 0;  // lanes past the last channel only take part in the group's maximum

    float2 w[W][2], bias[2];
    load_taps<W>(w, bias, a.w, a.bias, cc);
    const Rows<E, SRC8> rows(a, b, cc);
    const E* s0 = a.s0 ? static_cast<const E*>(a.s0) + (size_t)b * (W - 1) * a.D + cc : nullptr;
    E* y = static_cast<E*>(a.y) + (size_t)b * a.L * a.ldy + cc;
    const int ng = (a.D + 31) / 32;

    using R = Rows<E, SRC8>;
    typename R::Raw raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = t0 + u < t1 && cv ? rows.load(t0 + u) : R::zero();
    float2 x[W - 1 + U][2];  // x[W-1+u] is row t+u
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int t = t0 - (W - 1) + j;
        if (t < 0)
            past_row<E, W>(x[j], s0, t, a.D);
        else
            R::unpack(rows.load(t), x[j]);
    }
    for (int t = t0; t < t1; t += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            R::unpack(raw[u], x[W - 1 + u]);
            raw[u] = t + U + u < t1 && cv ? rows.load(t + U + u) : R::zero();
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u >= t1) break;
            float2 v[2];
            preact<W>(v, w, bias, &x[u]);
            if (SILU) silu4(v);
            if (cv) st_quad(y + (size_t)(t + u) * a.ldy, v);
            if (DST8) {
                float2 q[2] = {x[W - 1 + u][0], x[W - 1 + u][1]};
                const unsigned m = 0x7fffffffu;
                unsigned top = max(max(__float_as_uint(q[0].x) & m, __float_as_uint(q[0].y) & m),
                                   max(__float_as_uint(q[1].x) & m, __float_as_uint(q[1].y) & m));
                const unsigned grp = 0xffu << (threadIdx.x & 24);
                top = max(top, __shfl_xor_sync(grp, top, 1));
                top = max(top, __shfl_xor_sync(grp, top, 2));
                top = max(top, __shfl_xor_sync(grp, top, 4));
                const unsigned e = step_exponent(top);
                const size_t r = (size_t)b * a.L + t + u;
                if (cv) *reinterpret_cast<unsigned*>(a.q_out + r * a.D + c) = quantise4(q, e);
                if (cv && (c & 31) == 0) a.qe_out[r * ng + c / 32] = (uint8_t)e;
            }
        }
        if (t + U <= t1) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) { x[j][0] = x[U + j][0]; x[j][1] = x[U + j][1]; }
        }
    }
    if (a.sL && cv && t1 == a.L && seg == a.nseg - 1) {
        // the last W-1 inputs, read again: the window's place depends on the length
        E* sL = static_cast<E*>(a.sL) + (size_t)b * (W - 1) * a.D + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int t = a.L - (W - 1) + j;
            float2 v[2];
            if (t < 0)
                past_row<E, W>(v, s0, t, a.D);
            else
                R::unpack(rows.load(t), v);
            st_quad(sL + (size_t)j * a.D, v);
        }
    }
}

// ---------------------------------------------------------------- backward
// A piece's own rows t0..t1-1 give the sums of dw and dbias; dx_t needs g up to t + W-1, so the
// walk goes on for W-1 rows past the piece (g recomputed, not summed) and emits dx W-1 rows behind
// itself.  Past the end g is zero; before the start the rows are s0's.
template <typename E, int W, bool SILU, bool SRC8>
__global__ void __launch_bounds__(256, 2) conv_bwd_kernel(ConvArgs a) {
    __shared__ float red[256 * 4];
    const int tx = threadIdx.x % a.cx, ty = threadIdx.x / a.cx;
    const int64_t piece = (int64_t)blockIdx.x * a.ry + ty;
    const int c = (blockIdx.y * a.cx + tx) * 4;
    float2 sum[W + 1][2];
#pragma unroll
    for (int j = 0; j <= W; ++j) sum[j][0] = sum[j][1] = make_float2(0.f, 0.f);

    if (piece < (int64_t)a.B * a.nseg && c < a.D) {
        const int b = (int)(piece / a.nseg), seg = (int)(piece % a.nseg);
        const int t0 = seg * a.G, t1 = min(a.L, t0 + a.G);
        float2 w[W][2], bias[2];
        load_taps<W>(w, bias, a.w, a.bias, c);
        using R = Rows<E, SRC8>;
        const R rows(a, b, c);
        const size_t so = (size_t)b * (W - 1) * a.D + c;
        const E* s0 = a.s0 ? static_cast<const E*>(a.s0) + so : nullptr;
        const E* dsL = a.dsL ? static_cast<const E*>(a.dsL) + so : nullptr;
        E* ds0 = a.ds0 ? static_cast<E*>(a.ds0) + so : nullptr;
        const E* dy = static_cast<const E*>(a.dy) + (size_t)b * a.L * a.lddy + c;
        E* dx = static_cast<E*>(a.dx) + (size_t)b * a.L * a.lddx + c;
        const int tend = min(a.L, t1 + W - 1);  // rows with a gradient that this piece needs
        const int lo = t0 > 0 ? t0 : -(W - 1);  // rows whose gradient this piece writes: lo..t1-1

        typename R::Raw rx[U];
        typename Quad<E>::Raw rg[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            rx[u] = t0 + u < tend ? rows.load(t0 + u) : R::zero();
            rg[u] = t0 + u < tend ? ld_quad(dy + (size_t)(t0 + u) * a.lddy) : Quad<E>::zero();
        }
        float2 x[W - 1 + U][2];  // x[W-1+u] is row t+u
        float2 g[W - 1 + U][2];  // g[W-1+u] is row t+u
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int t = t0 - (W - 1) + j;
            if (t < 0)
                past_row<E, W>(x[j], s0, t, a.D);
            else
                R::unpack(rows.load(t), x[j]);
            g[j][0] = g[j][1] = make_float2(0.f, 0.f);
        }
        for (int t = t0; t < t1 + W - 1; t += U) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                R::unpack(rx[u], x[W - 1 + u]);
                Quad<E>::unpack(rg[u], g[W - 1 + u]);
                const int tn = t + U + u;
                rx[u] = tn < tend ? rows.load(tn) : R::zero();
                rg[u] = tn < tend ? ld_quad(dy + (size_t)tn * a.lddy) : Quad<E>::zero();
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float2 (&gu)[2] = g[W - 1 + u];  // dy, now to become dL/dv
                if (SILU) {
                    float2 v[2];
                    preact<W>(v, w, bias, &x[u]);
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const float2 s = make_float2(__fdividef(1.0f, 1.0f + ex2_mufu(-v[p].x * kLog2e)),
                                                     __fdividef(1.0f, 1.0f + ex2_mufu(-v[p].y * kLog2e)));
                        // d (v s) / dv = s + v s (1 - s)
                        const float2 one = make_float2(1.f, 1.f);
                        const float2 r = __ffma2_rn(s, make_float2(-1.f, -1.f), one);
                        gu[p] = __fmul2_rn(gu[p], __fmul2_rn(s, __ffma2_rn(v[p], r, one)));
                    }
                }
                if (t + u >= tend) gu[0] = gu[1] = make_float2(0.f, 0.f);
                if (t + u < t1) {
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
#pragma unroll
                        for (int j = 0; j < W; ++j) sum[j][p] = __ffma2_rn(gu[p], x[u + j][p], sum[j][p]);
                        sum[W][p] = __fadd2_rn(sum[W][p], gu[p]);
                    }
                }
                const int r = t + u - (W - 1);  // the row whose last contribution this is
                if (r < lo || r >= t1) continue;
                float2 d[2];
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    d[p] = __fmul2_rn(w[W - 1][p], g[u][p]);
#pragma unroll
                    for (int k = 1; k < W; ++k) d[p] = __ffma2_rn(w[W - 1 - k][p], g[u + k][p], d[p]);
                }
                if (dsL && r >= a.L - (W - 1)) {
                    float2 e[2];
                    Quad<E>::unpack(ld_quad(dsL + (size_t)(r - (a.L - (W - 1))) * a.D), e);
                    d[0] = __fadd2_rn(d[0], e[0]);
                    d[1] = __fadd2_rn(d[1], e[1]);
                }
                if (r >= 0)
                    st_quad(dx + (size_t)r * a.lddx, d);
                else if (ds0)
                    st_quad(ds0 + (size_t)(r + W - 1) * a.D, d);
            }
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                x[j][0] = x[U + j][0]; x[j][1] = x[U + j][1];
                g[j][0] = g[U + j][0]; g[j][1] = g[U + j][1];
            }
        }
    }
    // the CTA's sums over its ry pieces, in their order, one tap at a time
#pragma unroll 1
    for (int j = 0; j <= W; ++j) {
        float2 s[2] = {sum[0][0], sum[0][1]};
#pragma unroll
        for (int k = 1; k <= W; ++k)
            if (k == j) { s[0] = sum[k][0]; s[1] = sum[k][1]; }
        __syncthreads();
        *reinterpret_cast<float4*>(red + threadIdx.x * 4) = make_float4(s[0].x, s[0].y, s[1].x, s[1].y);
        __syncthreads();
        for (int i = threadIdx.x; i < a.cx * 4; i += blockDim.x) {
            const int ch = blockIdx.y * a.cx * 4 + i;
            if (ch >= a.D) continue;
            float v = 0.f;
            for (int k = 0; k < a.ry; ++k) v += red[k * a.cx * 4 + i];
            a.part[((size_t)blockIdx.x * (W + 1) + j) * a.D + ch] = v;
        }
    }
}

// dw and dbias from the CTAs' sums: 32 channels of one tap across, 8 shares of the CTAs down,
// added in a fixed order.
__global__ void __launch_bounds__(256) conv_reduce_kernel(const float* part, int parts, int D, int W,
                                                          float* dw, float* dbias) {
    __shared__ float red[8][32];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + tx, j = blockIdx.y;
    float s = 0.f;
    if (c < D)
        for (int k = ty; k < parts; k += 8) s += part[((size_t)k * (W + 1) + j) * D + c];
    red[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && c < D) {
#pragma unroll
        for (int k = 1; k < 8; ++k) s += red[k][tx];
        if (j < W)
            dw[(size_t)c * W + j] = s;
        else if (dbias)
            dbias[c] = s;
    }
}

// ---------------------------------------------------------------- packed prompts
// A row of threads takes one item (layer_common.cuh).  The state that a sequence starts from and
// the state that it leaves belong to the same pool entry: the thread that reads the old one (the
// sequence's first piece) also writes the new one, from x, so that no other thread of the launch
// touches the entry.
template <typename E, int W, bool SILU>
__global__ void __launch_bounds__(256) conv_prompt_kernel(ConvServeArgs a) {
    __shared__ int repeated[32];
    const int tx = threadIdx.x % a.cx, ty = threadIdx.x / a.cx;
    const int64_t item0 = (int64_t)blockIdx.x * a.ry, item = item0 + ty;
    if (threadIdx.x < 32) repeated[threadIdx.x] = 0;
    if (a.status && blockIdx.x == 0 && blockIdx.y == 0)
        check_batch(a.offsets, a.slot, a.S, a.rows, a.slots, a.rows, a.status);
    int s = find_seq(a.offsets, a.S, a.G, item0);
    for (int k = 0; k < ty && s + 1 < a.S && item_base(a.offsets, s + 1, a.G) <= item; ++k) ++s;
    const Span sp = item_span(a.offsets, a.slot, s, a.G, item, a.rows, a.slots, a.rows);
    __syncthreads();
    if (sp.ok && ty < a.ry && named_before(a.slot, sp.s, sp.slot, tx, a.cx)) repeated[ty] = 1;
    __syncthreads();
    if (!sp.ok || ty >= a.ry) return;
    if (repeated[ty]) {
        if (tx == 0) flag_if(a.status, kStatusInvalid);
        return;
    }
    const int c = (blockIdx.y * a.cx + tx) * 4;
    if (c >= a.D) return;
    const int t0 = sp.first, t1 = min(sp.end, t0 + a.G);
    const E* xr = static_cast<const E*>(a.x) + c;
    E* y = static_cast<E*>(a.y) + c;
    typename Quad<E>::Raw raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = t0 + u < t1 ? ld_quad(xr + (size_t)(t0 + u) * a.ldx) : Quad<E>::zero();
    float2 w[W][2], bias[2];
    load_taps<W>(w, bias, a.w, a.bias, c);
    float2 x[W - 1 + U][2];
    E* entry = sp.slot >= 0 ? static_cast<E*>(a.pool) + (size_t)sp.slot * (W - 1) * a.D + c : nullptr;
    if (sp.local == 0) {
        const bool carry = entry && a.carry && a.carry[sp.s];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            x[j][0] = x[j][1] = make_float2(0.f, 0.f);
            if (carry) Quad<E>::unpack(ld_quad(entry + (size_t)j * a.D), x[j]);
        }
        if (entry) {
            // entry i is input len + i - (W-1) of [past, x]: one of x, or of the W-1 in registers
            const int len = sp.end - t0;
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
                const int k = len + i;  // index into [past, x]
                float2 v[2] = {x[0][0], x[0][1]};
#pragma unroll
                for (int j = 1; j < W - 1; ++j)
                    if (k == j) { v[0] = x[j][0]; v[1] = x[j][1]; }
                if (k >= W - 1) Quad<E>::unpack(ld_quad(xr + (size_t)(t0 + k - (W - 1)) * a.ldx), v);
                st_quad(entry + (size_t)i * a.D, v);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            Quad<E>::unpack(ld_quad(xr + (size_t)(t0 - (W - 1) + j) * a.ldx), x[j]);
    }
    for (int t = t0; t < t1; t += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Quad<E>::unpack(raw[u], x[W - 1 + u]);
            raw[u] = t + U + u < t1 ? ld_quad(xr + (size_t)(t + U + u) * a.ldx) : Quad<E>::zero();
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u >= t1) break;
            float2 v[2];
            preact<W>(v, w, bias, &x[u]);
            if (SILU) silu4(v);
            st_quad(y + (size_t)(t + u) * a.ldy, v);
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) { x[j][0] = x[U + j][0]; x[j][1] = x[U + j][1]; }
    }
}

// ---------------------------------------------------------------- single tokens
// One row a CTA row: four channels a thread, every load issued before the first use.
template <typename E, int W, bool SILU>
__global__ void __launch_bounds__(256) conv_step_kernel(ConvServeArgs a) {
    const int row = blockIdx.y, c = (blockIdx.x * blockDim.x + threadIdx.x) * 4;
    const int k = a.slot ? a.slot[row] : row;
    const bool use = k >= 0 && k < a.slots;
    const bool work = use && c < a.D;
    E* entry = static_cast<E*>(a.pool) + (size_t)(use ? k : 0) * (W - 1) * a.D + c;
    typename Quad<E>::Raw raw[W];
#pragma unroll
    for (int j = 0; j < W; ++j) raw[j] = Quad<E>::zero();
    if (work) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) raw[j] = ld_quad(entry + (size_t)j * a.D);
        raw[W - 1] = ld_quad(static_cast<const E*>(a.x) + (size_t)row * a.ldx + c);
    }
    const bool repeated = a.slot && __syncthreads_or(named_before(a.slot, row, use ? k : -1, threadIdx.x, blockDim.x));
    if (k >= a.slots || repeated) {
        if (threadIdx.x == 0 && blockIdx.x == 0) flag_if(a.status, kStatusInvalid);
        return;
    }
    if (!work) return;
    float2 w[W][2], bias[2], x[W][2], v[2];
    load_taps<W>(w, bias, a.w, a.bias, c);
#pragma unroll
    for (int j = 0; j < W; ++j) Quad<E>::unpack(raw[j], x[j]);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        *reinterpret_cast<typename Quad<E>::Raw*>(entry + (size_t)j * a.D) = raw[j + 1];
    preact<W>(v, w, bias, x);
    if (SILU) silu4(v);
    st_quad(static_cast<E*>(a.y) + (size_t)row * a.ldy + c, v);
}

// ---------------------------------------------------------------- dispatch
// Calls f with the width, SiLU and element type as compile-time values.
template <int V> struct Int { static constexpr int value = V; };
template <typename E> struct Type { using type = E; };
template <typename F>
cudaError_t dispatch(int width, bool silu, int io_bf16, F f) {
    auto with_type = [&](auto w, auto s) {
        return io_bf16 ? f(Type<__nv_bfloat16>{}, w, s) : f(Type<float>{}, w, s);
    };
    auto with_silu = [&](auto w) {
        return silu ? with_type(w, Int<1>{}) : with_type(w, Int<0>{});
    };
    return width == 2 ? with_silu(Int<2>{}) : width == 3 ? with_silu(Int<3>{}) : with_silu(Int<4>{});
}

}  // namespace

// Rows a piece: enough pieces for about 1536 threads per SM, at least 8 rows (the W-1 rows before a
// piece are read twice) and at most 64.
int rows_per_piece(int64_t rows, int64_t D, int lo, int hi) {
    const int64_t g = rows * ((D + 31) / 32 * 8) / (148 * 1536);
    return (int)(g < lo ? lo : (g > hi ? hi : g));
}

}  // namespace conv

static void set_pieces(ConvArgs& a, int lo, int hi) {
    const conv::Tile t = conv::tile_of(a.D);
    a.cx = t.cx; a.ry = t.ry; a.nct = t.nct;
    const int G = conv::rows_per_piece((int64_t)a.B * a.L, a.D, lo, hi);
    a.nseg = a.L > 0 ? (a.L + G - 1) / G : 1;
    a.G = a.L > 0 ? (a.L + a.nseg - 1) / a.nseg : 1;
    a.nseg = a.L > 0 ? (a.L + a.G - 1) / a.G : 1;
    a.parts = (int)(((int64_t)a.B * a.nseg + t.ry - 1) / t.ry);
}
void conv_plan(ConvArgs& a, bool backward) {
    if (backward) set_pieces(a, 16, 64);
    else set_pieces(a, 8, 64);
}

cudaError_t launch_conv_fwd(const ConvArgs& a, int width, bool silu, int io_bf16, bool restore,
                            cudaStream_t st) {
    const dim3 grid(a.parts, a.nct), block(a.cx * a.ry);
    return conv::dispatch(width, silu, io_bf16, [&](auto e, auto w, auto s) {
        using E = typename decltype(e)::type;
        constexpr int W = decltype(w)::value;
        constexpr bool SL = decltype(s)::value != 0;
        if (restore)
            conv::conv_fwd_kernel<E, W, SL, true, false><<<grid, block, 0, st>>>(a);
        else if (a.q_out)
            conv::conv_fwd_kernel<E, W, SL, false, true><<<grid, block, 0, st>>>(a);
        else
            conv::conv_fwd_kernel<E, W, SL, false, false><<<grid, block, 0, st>>>(a);
        return cudaGetLastError();
    });
}

cudaError_t launch_conv_bwd(const ConvArgs& a, int width, bool silu, int io_bf16, cudaStream_t st) {
    const dim3 grid(a.parts, a.nct), block(a.cx * a.ry);
    cudaError_t e0 = conv::dispatch(width, silu, io_bf16, [&](auto e, auto w, auto s) {
        using E = typename decltype(e)::type;
        constexpr int W = decltype(w)::value;
        constexpr bool SL = decltype(s)::value != 0;
        if (a.q)
            conv::conv_bwd_kernel<E, W, SL, true><<<grid, block, 0, st>>>(a);
        else
            conv::conv_bwd_kernel<E, W, SL, false><<<grid, block, 0, st>>>(a);
        return cudaGetLastError();
    });
    if (e0 != cudaSuccess) return e0;
    conv::conv_reduce_kernel<<<dim3((a.D + 31) / 32, width + 1), 256, 0, st>>>(a.part, a.parts, a.D, width,
                                                                              a.dw, a.dbias);
    return cudaGetLastError();
}

cudaError_t launch_conv_prompt(ConvServeArgs a, int width, bool silu, int io_bf16, cudaStream_t st) {
    const conv::Tile t = conv::tile_of(a.D);
    a.cx = t.cx; a.ry = t.ry;
    a.G = conv::rows_per_piece(a.rows, a.D, 8, 64);
    a.items = (int64_t)(a.rows / a.G) + a.S;
    const dim3 grid((unsigned)((a.items + t.ry - 1) / t.ry), t.nct), block(256);  // whole warps
    return conv::dispatch(width, silu, io_bf16, [&](auto e, auto w, auto s) {
        using E = typename decltype(e)::type;
        conv::conv_prompt_kernel<E, decltype(w)::value, decltype(s)::value != 0><<<grid, block, 0, st>>>(a);
        return cudaGetLastError();
    });
}

cudaError_t launch_conv_step(const ConvServeArgs& a, int width, bool silu, int io_bf16, cudaStream_t st) {
    const int nvec = (a.D + 3) / 4;
    const int nt = nvec >= 256 ? 256 : (nvec + 31) / 32 * 32;
    const dim3 grid((nvec + nt - 1) / nt, a.rows), block(nt);
    return conv::dispatch(width, silu, io_bf16, [&](auto e, auto w, auto s) {
        using E = typename decltype(e)::type;
        conv::conv_step_kernel<E, decltype(w)::value, decltype(s)::value != 0><<<grid, block, 0, st>>>(a);
        return cudaGetLastError();
    });
}

}  // namespace ssm
