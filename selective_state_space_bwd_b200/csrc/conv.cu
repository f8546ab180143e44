// Short causal convolution in front of the scan: forward, its recomputation from an 8-bit
// checkpoint, its gradient, and the packed-prompt and single-token forms (include/ssm_scan.h).
//
// The plain forward and the gradient run at 85 to 90 % of the copy bandwidth on large inputs.  The 8-bit forms in
// bf16 (60 to 77 %; in fp32 80 to 85 %) issue an instruction in half of the cycles at 14 warps an SM, and wait for the
// latency of the ones before it (SiLU, conversion, W products).  A thread owns V consecutive
// channels and walks down a piece of the rows, the last W-1 inputs in registers, so that an element
// is read once from DRAM (the W-1 rows before a piece a second time).  Each thread copies its
// own rows into its own places of a ring in shared memory, kDepth - 1 groups of four rows ahead
// (cp.async, 16 or 8 bytes): the bytes in flight, 32 to 64 KB an SM, cost no registers, and since no other
// thread reads them there is no barrier in the loop, only the thread's own wait_group.
//
// A CTA is cx threads across (a multiple of the 32 / V threads that share an 8-bit group's 32 channels, so
// that they are neighbours in a warp) by ry pieces down; the channels are cut into equal tiles of at most
// 32 threads, so that a width just past a tile leaves no tile empty.  The pieces are as long as one
// wave of CTAs allows: long pieces read fewer rows twice and, in the gradient, leave fewer sums.
#include "layer_common.cuh"
#include "real_common.cuh"

#include <type_traits>

namespace ssm {
namespace conv {
namespace {

constexpr int kThreads = 256;
constexpr int kResident = 296;   // CTAs of a wave: two per SM (registers, and the ring)
constexpr int U = 4;             // rows a group; row t of a piece that starts at t0 lies in slot (t - t0) % 4

using real::cp_async;
using real::cp_async_commit;
using real::cp_async_wait;

struct Tile {
    int cx, ry, nct;
};
Tile tile_of(int D, int V) {
    const int grp = 32 / V;  // threads of 32 channels
    const int nvec = (D + 31) / 32 * grp;
    Tile t;
    t.nct = (nvec + 31) / 32;
    t.cx = ((nvec + t.nct - 1) / t.nct + grp - 1) / grp * grp;
    t.ry = kThreads / t.cx;
    return t;
}

// The taps of V channels, tap-major: w[j][pair].
template <int W, int V>
__device__ __forceinline__ void load_taps(float2 (&w)[W][V / 2], float2 (&bias)[V / 2], const float* pw,
                                          const float* pb, int c) {
    float f[V * W];
#pragma unroll
    for (int i = 0; i < V * W / 4; ++i) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(pw + (size_t)c * W) + i);
        f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
    }
#pragma unroll
    for (int p = 0; p < V / 2; ++p) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][p] = make_float2(f[2 * p * W + j], f[(2 * p + 1) * W + j]);
        bias[p] = pb ? __ldg(reinterpret_cast<const float2*>(pb + c) + p) : make_float2(0.f, 0.f);
    }
}

// The pre-activation of the row in slot u from the rows in the slots before it.  (Taps scaled by log2 e, which
// would spare SiLU the product in front of its exp2, took 376 us against 381 for the training calls at 4 x 8192 x
// 4096 from 8 bits.  They were taken out: a finite pre-activation past 2.36e38 became infinite, its gradient NaN.)
template <int W, int P>
__device__ __forceinline__ void preact(float2 (&v)[P], const float2 (&w)[W][P], const float2 (&bias)[P],
                                       const float2 (&x)[U][P], int u) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
        v[p] = bias[p];
#pragma unroll
        for (int j = 0; j < W; ++j) v[p] = __ffma2_rn(w[j][p], x[(u + U - (W - 1) + j) % U][p], v[p]);
    }
}

template <int P>
__device__ __forceinline__ void silu(float2 (&v)[P]) {
#pragma unroll
    for (int p = 0; p < P; ++p) v[p] = silu_pair(v[p]);
}

// ---------------------------------------------------------------- 8-bit checkpoint
// The step of magnitudes from 2^127 on: 64 of twice that would be 2^128, so there 127 steps are
// the limit instead.
constexpr unsigned kTopStep = 248u;

// The biased exponent of a group's step from the largest magnitude's bits (an unsigned maximum, so
// that a NaN, above every number's bits, is not lost as fmaxf would lose it).
// 127.5 / 64 has the mantissa 0x7f0000, so that adding 2^16 carries into the exponent from there on.
__device__ __forceinline__ unsigned step_exponent(unsigned top) {
    unsigned q = min(max((top + 0x10000u) >> 23, 7u) - 6u, kTopStep);
    if (top == 0u) q = 0u;
    if (top >= 0x7f800000u) q = 255u;
    return q;
}

// The largest magnitude of V channels, as fp32 bits; bf16 pairs are compared as they lie in the row.
template <typename E, int P>
__device__ __forceinline__ unsigned top_of(const float2 (&x)[P]) {
    unsigned m[P];
    if constexpr (sizeof(E) == 2) {
#pragma unroll
        for (int p = 0; p < P; ++p)
            m[p] = __byte_perm(__float_as_uint(x[p].x), __float_as_uint(x[p].y), 0x7632) & 0x7fff7fffu;
#pragma unroll
        for (int p = 1; p < P; ++p) m[0] = __vmaxu2(m[0], m[p]);
        return max(m[0] << 16, m[0] & 0xffff0000u);
    } else {
#pragma unroll
        for (int p = 0; p < P; ++p)
            m[p] = max(__float_as_uint(x[p].x) & 0x7fffffffu, __float_as_uint(x[p].y) & 0x7fffffffu);
#pragma unroll
        for (int p = 1; p < P; ++p) m[0] = max(m[0], m[p]);
        return m[0];
    }
}

// Four int8 of x / 2^(qe - 127), rounded to nearest even: adding 1.5 * 2^23 leaves the rounded
// integer in the low bits of the sum (the product by a power of two is exact).
__device__ __forceinline__ unsigned quantise4(float2 x0, float2 x1, unsigned qe) {
    const float f = __uint_as_float((254u - qe) << 23);  // a normal number; zeros (qe 0) stay zeros
    if (qe >= kTopStep) {
        if (qe == 255u) return 0u;
        const float m = 127.0f * __uint_as_float(kTopStep << 23);
        x0 = make_float2(fminf(fmaxf(x0.x, -m), m), fminf(fmaxf(x0.y, -m), m));
        x1 = make_float2(fminf(fmaxf(x1.x, -m), m), fminf(fmaxf(x1.y, -m), m));
    }
    const float magic = 12582912.0f;
    const float2 a = __ffma2_rn(x0, make_float2(f, f), make_float2(magic, magic));
    const float2 b = __ffma2_rn(x1, make_float2(f, f), make_float2(magic, magic));
    const unsigned lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
    const unsigned hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}

// The values of four int8.  A byte u = q + 128 in the low bits of 2^23 is the float 2^23 + u; the
// step of a NaN group (exponent 255) is infinite and its q zero, and 0 * inf is the NaN wanted.
__device__ __forceinline__ void restore4(float2& x0, float2& x1, unsigned q, unsigned qe) {
    const float step = __uint_as_float(qe << 23);
    const unsigned u = q ^ 0x80808080u;
    const float off = -8388736.0f;  // -(2^23 + 128)
    const float2 o = make_float2(off, off), s = make_float2(step, step);
    const float2 a = make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540)),
                                 __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7541)));
    const float2 b = make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7542)),
                                 __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7543)));
    x0 = __fmul2_rn(__fadd2_rn(a, o), s);
    x1 = __fmul2_rn(__fadd2_rn(b, o), s);
}

// ---------------------------------------------------------------- row sources
// Rows of V channels of one batch entry, from x or from its 8-bit checkpoint.  word(t): the step
// exponents of the four rows from t on (t a multiple of four), a byte a row; unused for x.
template <typename E, int V, bool Q8> struct Rows;
template <typename E, int V> struct Rows<E, V, false> {
    using Raw = typename Vec<E, V>::Raw;
    const E* x;
    unsigned ldb;
    __device__ __forceinline__ Rows(const ConvArgs& a, int b, int c)
        : x(static_cast<const E*>(a.x) + (size_t)b * a.L * a.ldx + c), ldb((unsigned)(a.ldx * sizeof(E))) {}
    __device__ __forceinline__ const void* at(int t) const { return row_at(x, t, ldb); }
    __device__ __forceinline__ unsigned word(int) const { return 0u; }
    static __device__ __forceinline__ void unpack(const Raw& r, unsigned, float2 (&o)[V / 2]) {
        Vec<E, V>::unpack(r, o);
    }
    __device__ __forceinline__ void load(int t, float2 (&o)[V / 2]) const {
        Vec<E, V>::unpack(*static_cast<const Raw*>(at(t)), o);
    }
};
template <typename E> struct Rows<E, 4, true> {
    using Raw = unsigned;
    const int8_t* q;
    const uint8_t* e;
    unsigned ldb;  // D
    __device__ __forceinline__ Rows(const ConvArgs& a, int b, int c)
        : q(a.q + (size_t)b * a.L * a.D + c),
          e(a.qe + ((size_t)b * ((a.D + 31) / 32) + c / 32) * a.Lq), ldb((unsigned)a.D) {}
    __device__ __forceinline__ const void* at(int t) const { return row_at(q, t, ldb); }
    __device__ __forceinline__ unsigned word(int t) const { return *reinterpret_cast<const unsigned*>(e + t); }
    static __device__ __forceinline__ void unpack(const Raw& r, unsigned e, float2 (&o)[2]) {
        restore4(o[0], o[1], r, e);
    }
    __device__ __forceinline__ void load(int t, float2 (&o)[2]) const {
        restore4(o[0], o[1], *static_cast<const Raw*>(at(t)), e[t]);
    }
};
template <typename E> struct Rows<E, 8, true> {
    using Raw = uint2;
    const int8_t* q;
    const uint8_t* e;
    unsigned ldb;  // D
    __device__ __forceinline__ Rows(const ConvArgs& a, int b, int c)
        : q(a.q + (size_t)b * a.L * a.D + c),
          e(a.qe + ((size_t)b * ((a.D + 31) / 32) + c / 32) * a.Lq), ldb((unsigned)a.D) {}
    __device__ __forceinline__ const void* at(int t) const { return row_at(q, t, ldb); }
    __device__ __forceinline__ unsigned word(int t) const { return *reinterpret_cast<const unsigned*>(e + t); }
    static __device__ __forceinline__ void unpack(const Raw& r, unsigned e, float2 (&o)[4]) {
        restore4(o[0], o[1], r.x, e);
        restore4(o[2], o[3], r.y, e);
    }
    __device__ __forceinline__ void load(int t, float2 (&o)[4]) const {
        unpack(*static_cast<const Raw*>(at(t)), e[t], o);
    }
};

// Row t < 0 of a sequence: the state before it, or zero.
template <typename E, int W, int V>
__device__ __forceinline__ void past_row(float2 (&o)[V / 2], const E* s0, int t, size_t D) {
    if (s0) {
        Vec<E, V>::unpack(ld_vec<E, V>(s0 + (size_t)(t + W - 1) * D), o);
    } else {
#pragma unroll
        for (int p = 0; p < V / 2; ++p) o[p] = make_float2(0.f, 0.f);
    }
}

// ---------------------------------------------------------------- forward
// SRC8: from the checkpoint (restore); DST8: write the checkpoint.
template <typename E, int V, int W, bool SILU, bool SRC8, bool DST8>
struct Fwd {
    using R = Rows<E, V, SRC8>;
    // Groups in the ring: one or two on their way.  Bytes in flight are not what the forward waits for: at
    // 4 x 8192 x 4096 it takes 92 us with one group of 16-byte rows ahead, 103 with two to four.
    static constexpr int kDepth = sizeof(typename R::Raw) == 16 ? 2 : 3;
    static constexpr int kBytes = kDepth * U * kThreads * (int)sizeof(typename R::Raw);
};

template <typename E, int V, int W, bool SILU, bool SRC8, bool DST8>
__global__ void __launch_bounds__(kThreads, 2) conv_fwd_kernel(ConvArgs a) {
    using F = Fwd<E, V, W, SILU, SRC8, DST8>;
    using R = typename F::R;
    using Raw = typename R::Raw;
    constexpr int P = V / 2, DEPTH = F::kDepth;
    extern __shared__ __align__(16) unsigned char smem[];
    Raw* ring = reinterpret_cast<Raw*>(smem) + threadIdx.x;  // slot k: ring[k * kThreads]
    const int tx = threadIdx.x % a.cx, ty = threadIdx.x / a.cx;
    const int64_t piece = (int64_t)blockIdx.x * a.ry + ty;
    if (ty >= a.ry || piece >= (int64_t)a.B * a.nseg) return;  // whole rows of threads: whole 8-bit groups
    const int c = (blockIdx.y * a.cx + tx) * V;
    const bool cv = c < a.D;
    const int b = (int)(piece / a.nseg), seg = (int)(piece % a.nseg);
    const int t0 = seg * a.G, t1 = min(a.L, t0 + a.G);
    if (!DST8 && !cv) return;
    const int cc = cv ? c : 0;  // lanes past the last channel only take part in the group's maximum

    const R rows(a, b, cc);
    auto issue = [&](int t, int stage) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t + u < t1) cp_async<sizeof(Raw)>(ring + (stage * U + u) * kThreads, rows.at(t + u));
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < DEPTH - 1; ++s) issue(t0 + s * U, s);
    unsigned ew = SRC8 && t0 < t1 ? rows.word(t0) : 0u;

    float2 w[W][P], bias[P], x[U][P];
    load_taps<W, V>(w, bias, a.w, a.bias, cc);
    const E* s0 = a.s0 ? static_cast<const E*>(a.s0) + (size_t)b * (W - 1) * a.D + cc : nullptr;
#pragma unroll
    for (int j = 1; j < W; ++j) {
        if (t0 - j < 0)
            past_row<E, W, V>(x[U - j], s0, t0 - j, a.D);
        else
            rows.load(t0 - j, x[U - j]);
    }
    E* y = static_cast<E*>(a.y) + (size_t)b * a.L * a.ldy + cc;
    const unsigned ldyb = (unsigned)(a.ldy * sizeof(E));
    int8_t* qo = DST8 ? a.q_out + (size_t)b * a.L * a.D + cc : nullptr;
    int stage = 0;
    for (int t = t0; t < t1; t += U) {
        issue(t + (DEPTH - 1) * U, stage == 0 ? DEPTH - 1 : stage - 1);
        unsigned en = 0u;
        if (SRC8 && t + U < t1) en = rows.word(t + U);
        cp_async_wait<DEPTH - 1>();
        unsigned steps = 0u;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u >= t1) break;
            R::unpack(ring[(stage * U + u) * kThreads], __byte_perm(ew, 0u, 0x4440 | u), x[u]);
            float2 v[P];
            preact<W, P>(v, w, bias, x, u);
            if (SILU) silu<P>(v);
            if (cv) st_vec<E, V>(row_at(y, t + u, ldyb), v);
            if (DST8) {
                unsigned top = cv ? top_of<E, P>(x[u]) : 0u;
                constexpr int GL = 32 / V;  // lanes of a group
                const unsigned grp = ((1u << GL) - 1u) << (threadIdx.x & (32 - GL));
#pragma unroll
                for (int m = 1; m < GL; m <<= 1) top = max(top, __shfl_xor_sync(grp, top, m));
                const unsigned e = step_exponent(top);
                steps |= e << (8 * u);
                if (cv) {
                    if constexpr (V == 4)
                        *reinterpret_cast<unsigned*>(row_at(qo, t + u, a.D)) = quantise4(x[u][0], x[u][1], e);
                    else
                        *reinterpret_cast<uint2*>(row_at(qo, t + u, a.D)) =
                            make_uint2(quantise4(x[u][0], x[u][1], e), quantise4(x[u][P - 2], x[u][P - 1], e));
                }
            }
        }
        if (DST8 && cv && (c & 31) == 0)
            *reinterpret_cast<unsigned*>(a.qe_out + ((size_t)b * ((a.D + 31) / 32) + c / 32) * a.Lq + t) = steps;
        ew = en;
        stage = stage == DEPTH - 1 ? 0 : stage + 1;
    }
    if (a.sL && cv && seg == a.nseg - 1) {
        // the last W-1 inputs, read again: the window's place depends on the length
        E* sL = static_cast<E*>(a.sL) + (size_t)b * (W - 1) * a.D + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int t = a.L - (W - 1) + j;
            float2 v[P];
            if (t < 0)
                past_row<E, W, V>(v, s0, t, a.D);
            else
                rows.load(t, v);
            st_vec<E, V>(sL + (size_t)j * a.D, v);
        }
    }
}

// ---------------------------------------------------------------- backward
// A piece's own rows t0..t1-1 give the sums of dw and dbias; dx_t needs g up to t + W-1, so the
// walk goes on for W-1 rows past the piece (g recomputed, not summed) and emits dx W-1 rows behind
// itself.  Past the end g is zero; before the start the rows are s0's.  Four channels a thread: W
// taps, W+1 sums and the two windows are 60 registers, and two CTAs stay resident.
template <typename E, bool SRC8>
struct Bwd {
    using R = Rows<E, 4, SRC8>;
    using Raw = typename R::Raw;
    using GRaw = typename Vec<E, 4>::Raw;
    static constexpr int kPer = U * kThreads * (int)(sizeof(Raw) + sizeof(GRaw));
    static constexpr int kDepth = kPer <= 12288 ? 4 : (kPer <= 16384 ? 3 : 2);
    static constexpr int kBytes = kDepth * kPer;  // the sums at the end, 20 KB, reuse it
};

template <typename E, int W, bool SILU, bool SRC8>
__global__ void __launch_bounds__(kThreads, 2) conv_bwd_kernel(ConvArgs a) {
    using Cfg = Bwd<E, SRC8>;
    using R = typename Cfg::R;
    using Raw = typename Cfg::Raw;
    using GRaw = typename Cfg::GRaw;
    constexpr int DEPTH = Cfg::kDepth;
    extern __shared__ __align__(16) unsigned char smem[];
    GRaw* gring = reinterpret_cast<GRaw*>(smem) + threadIdx.x;
    Raw* xring = reinterpret_cast<Raw*>(smem + DEPTH * U * kThreads * sizeof(GRaw)) + threadIdx.x;
    const int tx = threadIdx.x % a.cx, ty = threadIdx.x / a.cx;
    const int64_t piece = (int64_t)blockIdx.x * a.ry + ty;
    const int c = (blockIdx.y * a.cx + tx) * 4;
    float2 sum[W + 1][2];
#pragma unroll
    for (int j = 0; j <= W; ++j) sum[j][0] = sum[j][1] = make_float2(0.f, 0.f);

    if (ty < a.ry && piece < (int64_t)a.B * a.nseg && c < a.D) {
        const int b = (int)(piece / a.nseg), seg = (int)(piece % a.nseg);
        const int t0 = seg * a.G, t1 = min(a.L, t0 + a.G);
        const int tend = min(a.L, t1 + W - 1);  // rows with a gradient that this piece needs
        const int lo = t0 > 0 ? t0 : -(W - 1);  // rows whose gradient this piece writes: lo..t1-1
        const R rows(a, b, c);
        const E* dy = static_cast<const E*>(a.dy) + (size_t)b * a.L * a.lddy + c;
        const unsigned lddyb = (unsigned)(a.lddy * sizeof(E)), lddxb = (unsigned)(a.lddx * sizeof(E));
        // Rows are issued in order, so their addresses are running sums (one addition a row instead of a
        // wide product: 152 -> 146 us at 4 x 8192 x 4096, 173 -> 168 from 8 bits).
        uintptr_t gp = (uintptr_t)row_at(dy, t0, lddyb), xp = (uintptr_t)rows.at(t0);
        auto issue = [&](int t, int stage) {
            auto one = [&](int u, bool there) {
                if (there) {
                    cp_async<sizeof(GRaw)>(gring + (stage * U + u) * kThreads, (const void*)gp);
                    cp_async<sizeof(Raw)>(xring + (stage * U + u) * kThreads, (const void*)xp);
                }
                gp += lddyb;
                xp += rows.ldb;
            };
            if (t + U <= tend) {
#pragma unroll
                for (int u = 0; u < U; ++u) one(u, true);
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) one(u, t + u < tend);
            }
            cp_async_commit();
        };
#pragma unroll
        for (int s = 0; s < DEPTH - 1; ++s) issue(t0 + s * U, s);
        unsigned ew = SRC8 && t0 < tend ? rows.word(t0) : 0u;

        float2 w[W][2], bias[2], x[U][2], g[U][2];
        load_taps<W, 4>(w, bias, a.w, a.bias, c);
        const size_t so = (size_t)b * (W - 1) * a.D + c;
        const E* s0 = a.s0 ? static_cast<const E*>(a.s0) + so : nullptr;
        const E* dsL = a.dsL ? static_cast<const E*>(a.dsL) + so : nullptr;
        E* ds0 = a.ds0 ? static_cast<E*>(a.ds0) + so : nullptr;
        E* dx = static_cast<E*>(a.dx) + (size_t)b * a.L * a.lddx + c;
#pragma unroll
        for (int j = 1; j < W; ++j) {
            if (t0 - j < 0)
                past_row<E, W, 4>(x[U - j], s0, t0 - j, a.D);
            else
                rows.load(t0 - j, x[U - j]);
            g[U - j][0] = g[U - j][1] = make_float2(0.f, 0.f);
        }
        uintptr_t dp = (uintptr_t)dx + (unsigned long long)t0 * lddxb - (unsigned long long)(W - 1) * lddxb;
        // one row: INNER when it is summed, writes a row of dx, and nothing touches the ends
        auto row = [&](int t, int u, int stage, auto inner) {
            constexpr bool INNER = decltype(inner)::value;
            R::unpack(xring[(stage * U + u) * kThreads], __byte_perm(ew, 0u, 0x4440 | u), x[u]);
            Vec<E, 4>::unpack(gring[(stage * U + u) * kThreads], g[u]);  // dy, now to become dL/dv
            if (SILU) {
                float2 v[2];
                preact<W, 2>(v, w, bias, x, u);
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    // d (v s) / dv = s (1 + v (1 - s)).  Of v from 18 on s is one to the bit, so that the difference
                    // is zero however large v is.
                    const float2 one = make_float2(1.f, 1.f);
                    const float2 s = sigmoid_pair(v[p]);
                    const float2 r = __ffma2_rn(s, make_float2(-1.f, -1.f), one);
                    g[u][p] = __fmul2_rn(g[u][p], __fmul2_rn(s, __ffma2_rn(v[p], r, one)));
                }
            }
            if (!INNER && t >= tend) g[u][0] = g[u][1] = make_float2(0.f, 0.f);  // the ring holds other rows
            if (INNER || t < t1) {
#pragma unroll
                for (int p = 0; p < 2; ++p) {
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        sum[j][p] = __ffma2_rn(g[u][p], x[(u + U - (W - 1) + j) % U][p], sum[j][p]);
                    sum[W][p] = __fadd2_rn(sum[W][p], g[u][p]);
                }
            }
            const int r = t - (W - 1);  // the row whose last contribution this is
            if (!INNER && (r < lo || r >= t1)) return;
            float2 d[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                d[p] = __fmul2_rn(w[W - 1][p], g[(u + U - (W - 1)) % U][p]);
#pragma unroll
                for (int k = 1; k < W; ++k)
                    d[p] = __ffma2_rn(w[W - 1 - k][p], g[(u + U - (W - 1) + k) % U][p], d[p]);
            }
            if (!INNER && dsL && r >= a.L - (W - 1)) {
                float2 e[2];
                Vec<E, 4>::unpack(ld_vec<E, 4>(dsL + (size_t)(r - (a.L - (W - 1))) * a.D), e);
                d[0] = __fadd2_rn(d[0], e[0]);
                d[1] = __fadd2_rn(d[1], e[1]);
            }
            if (INNER || r >= 0)
                st_vec<E, 4>(reinterpret_cast<E*>(dp + (unsigned long long)u * lddxb), d);
            else if (ds0)
                st_vec<E, 4>(ds0 + (size_t)(r + W - 1) * a.D, d);
        };
        int stage = 0;
        for (int t = t0; t < t1 + W - 1; t += U) {
            issue(t + (DEPTH - 1) * U, stage == 0 ? DEPTH - 1 : stage - 1);
            unsigned en = 0u;
            if (SRC8 && t + U < tend) en = rows.word(t + U);
            cp_async_wait<DEPTH - 1>();
            if (t > t0 && t + U <= t1) {
#pragma unroll
                for (int u = 0; u < U; ++u) row(t + u, u, stage, std::true_type{});
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) row(t + u, u, stage, std::false_type{});
            }
            ew = en;
            dp += (unsigned long long)U * lddxb;
            stage = stage == DEPTH - 1 ? 0 : stage + 1;
        }
    }
    // the CTA's sums over its ry pieces, in their order
    cp_async_wait<0>();
    __syncthreads();
    float* red = reinterpret_cast<float*>(smem);  // [W+1][ry][cx * 4]
    const int wid = a.cx * 4;
    if (ty < a.ry) {
#pragma unroll
        for (int j = 0; j <= W; ++j)
            *reinterpret_cast<float4*>(red + (j * a.ry + ty) * wid + tx * 4) =
                make_float4(sum[j][0].x, sum[j][0].y, sum[j][1].x, sum[j][1].y);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (W + 1) * wid; i += kThreads) {
        const int j = i / wid, k = i - j * wid, ch = blockIdx.y * wid + k;
        if (ch >= a.D) continue;
        float v = 0.f;
        for (int r = 0; r < a.ry; ++r) v += red[(j * a.ry + r) * wid + k];
        a.part[((size_t)blockIdx.x * (W + 1) + j) * a.D + ch] = v;
    }
}

// dw and dbias from the CTAs' sums: 32 channels of one tap across, 8 shares of the CTAs down,
// added in a fixed order.  Its first thread writes the status word: nothing in the gradient can
// fail on the device.
__global__ void __launch_bounds__(256) conv_reduce_kernel(const float* part, int parts, int D, int W,
                                                          float* dw, float* dbias, unsigned* status) {
    __shared__ float red[8][32];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + tx, j = blockIdx.y;
    if (blockIdx.x == 0 && j == 0 && threadIdx.x == 0) *status = 0u;
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
template <typename E, int V, int W, bool SILU>
__global__ void __launch_bounds__(kThreads, 2) conv_prompt_kernel(ConvServeArgs a) {
    using Raw = typename Vec<E, V>::Raw;
    constexpr int P = V / 2, DEPTH = Fwd<E, V, W, SILU, false, false>::kDepth;
    extern __shared__ __align__(16) unsigned char smem[];
    Raw* ring = reinterpret_cast<Raw*>(smem) + threadIdx.x;
    __shared__ int repeated[kThreads / 4 + 1];
    const int tx = threadIdx.x % a.cx, ty = threadIdx.x / a.cx;
    const int64_t item0 = (int64_t)blockIdx.x * a.ry, item = item0 + ty;
    if (threadIdx.x <= kThreads / 4) repeated[threadIdx.x] = 0;
    if (a.status && blockIdx.x == 0 && blockIdx.y == 0)
        check_batch(a.offsets, a.slot, a.S, a.rows, a.slots, a.rows, a.status);
    int s = find_seq(a.offsets, a.S, a.G, item0);
    for (int k = 0; k < ty && s + 1 < a.S && item_base(a.offsets, s + 1, a.G) <= item; ++k) ++s;
    const bool carried = a.carry && a.carry[s];  // on its way together with the offsets
    const Span sp = item_span(a.offsets, a.slot, s, a.G, item, a.rows, a.slots);
    __syncthreads();
    if (sp.ok && ty < a.ry && named_before(a.slot, sp.s, sp.slot, tx, a.cx)) repeated[ty] = 1;
    __syncthreads();
    if (!sp.ok || ty >= a.ry) return;
    if (repeated[ty]) {
        if (tx == 0) flag_if(a.status, kStatusInvalid);
        return;
    }
    const int c = (blockIdx.y * a.cx + tx) * V;
    if (c >= a.D) return;
    const int t0 = sp.first, t1 = min(sp.end, t0 + a.G);
    const E* xr = static_cast<const E*>(a.x) + c;
    const unsigned ldxb = (unsigned)(a.ldx * sizeof(E)), ldyb = (unsigned)(a.ldy * sizeof(E));
    auto issue = [&](int t, int stage) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t + u < t1) cp_async<sizeof(Raw)>(ring + (stage * U + u) * kThreads, row_at(xr, t + u, ldxb));
        cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < DEPTH - 1; ++k) issue(t0 + k * U, k);
    float2 w[W][P], bias[P], x[U][P];
    load_taps<W, V>(w, bias, a.w, a.bias, c);
    E* entry = sp.slot >= 0 ? static_cast<E*>(a.pool) + (size_t)sp.slot * (W - 1) * a.D + c : nullptr;
    if (sp.local == 0) {
        const bool carry = entry && carried;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {  // entry j is input j - (W-1): slot U - (W-1) + j
            float2 (&o)[P] = x[U - (W - 1) + j];
#pragma unroll
            for (int p = 0; p < P; ++p) o[p] = make_float2(0.f, 0.f);
            if (carry) Vec<E, V>::unpack(ld_vec<E, V>(entry + (size_t)j * a.D), o);
        }
        if (entry) {
            // entry i becomes input len + i of [past, x]: one of x, or one of the W-1 in registers
            const int len = sp.end - t0;
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
                const int k = len + i;
                float2 v[P];
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    v[p] = x[U - (W - 1)][p];
#pragma unroll
                    for (int j = 1; j < W - 1; ++j)
                        if (k == j) v[p] = x[U - (W - 1) + j][p];
                }
                if (k >= W - 1) Vec<E, V>::unpack(ld_vec<E, V>(xr + (size_t)(t0 + k - (W - 1)) * a.ldx), v);
                st_vec<E, V>(entry + (size_t)i * a.D, v);
            }
        }
    } else {
#pragma unroll
        for (int j = 1; j < W; ++j) Vec<E, V>::unpack(ld_vec<E, V>(xr + (size_t)(t0 - j) * a.ldx), x[U - j]);
    }
    E* y = static_cast<E*>(a.y) + c;
    int stage = 0;
    for (int t = t0; t < t1; t += U) {
        issue(t + (DEPTH - 1) * U, stage == 0 ? DEPTH - 1 : stage - 1);
        cp_async_wait<DEPTH - 1>();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u >= t1) break;
            Vec<E, V>::unpack(ring[(stage * U + u) * kThreads], x[u]);
            float2 v[P];
            preact<W, P>(v, w, bias, x, u);
            if (SILU) silu<P>(v);
            st_vec<E, V>(row_at(y, t + u, ldyb), v);
        }
        stage = stage == DEPTH - 1 ? 0 : stage + 1;
    }
}

// ---------------------------------------------------------------- single tokens
// Four channels a thread and R rows a CTA: the taps, as many bytes as a row's state and input in bf16, are read
// once for the R rows, whose states are on their way together.
template <typename E, int W, bool SILU, int R>
__global__ void __launch_bounds__(256) conv_step_kernel(ConvServeArgs a) {
    using Raw = typename Vec<E, 4>::Raw;
    const int row0 = blockIdx.y * R, c = (blockIdx.x * blockDim.x + threadIdx.x) * 4;
    const bool cv = c < a.D;
    int k[R];
#pragma unroll
    for (int r = 0; r < R; ++r) k[r] = row0 + r < a.rows ? (a.slot ? a.slot[row0 + r] : row0 + r) : -1;
    Raw raw[R][W];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool work = cv && k[r] >= 0 && k[r] < a.slots;
        const E* entry = static_cast<const E*>(a.pool) + (size_t)(work ? k[r] : 0) * (W - 1) * a.D + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) raw[r][j] = work ? ld_vec<E, 4>(entry + (size_t)j * a.D) : Vec<E, 4>::zero();
        raw[r][W - 1] = work ? ld_vec<E, 4>(static_cast<const E*>(a.x) + (size_t)(row0 + r) * a.ldx + c)
                             : Vec<E, 4>::zero();
    }
    float2 w[W][2], bias[2];
    load_taps<W, 4>(w, bias, a.w, a.bias, cv ? c : 0);
    if (a.slot) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = k[r] >= 0 && k[r] < a.slots;
            const bool rep = __syncthreads_or(named_before(a.slot, row0 + r, in ? k[r] : -1, threadIdx.x, blockDim.x));
            if (rep || k[r] >= a.slots) {
                if (threadIdx.x == 0 && blockIdx.x == 0) flag_if(a.status, kStatusInvalid);
                k[r] = -1;
            }
        }
    }
    if (!cv) return;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (k[r] < 0) continue;
        float2 x[U][2], v[2];
#pragma unroll
        for (int j = 0; j < W; ++j) Vec<E, 4>::unpack(raw[r][j], x[U - W + j]);
        E* entry = static_cast<E*>(a.pool) + (size_t)k[r] * (W - 1) * a.D + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) *reinterpret_cast<Raw*>(entry + (size_t)j * a.D) = raw[r][j + 1];
        preact<W, 2>(v, w, bias, x, U - 1);
        if (SILU) silu<2>(v);
        st_vec<E, 4>(static_cast<E*>(a.y) + (size_t)(row0 + r) * a.ldy + c, v);
    }
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

// Rows a piece of one batch entry: as many as give one wave of CTAs, at least 8 (the W-1 rows before a
// piece are read twice) and at most 512 (the gradient adds a piece's rows one after another in fp32;
// then a CTA its ry <= 64 pieces, and the reduction an eighth of the
// CTAs' sums and eight more, so that a sum is a chain of 512 + 64 + parts / 8 + 8 additions at most: 900 at
// 32768 rows x 4096 channels).  A multiple of four: a word of step exponents.
// `extra` pieces of the wave are kept free (a packed batch has up to one partly empty piece a sequence).
int rows_per_piece(int64_t batch, int64_t rows, const Tile& t, int64_t extra) {
    if (batch < 1) batch = 1;
    int64_t room = (int64_t)(kResident / t.nct) * t.ry;  // pieces of one channel tile in a wave
    if (extra) room = room > 2 * extra ? room - extra : room / 2;
    int64_t n = room / batch;
    if (n < 4) n = 4 * room / batch;  // too few per entry to fill a wave evenly: shorter pieces, more waves
    if (n < 1) n = 1;
    int64_t g = ((rows + n - 1) / n + 3) / 4 * 4;
    return (int)(g < 8 ? 8 : (g > 512 ? 512 : g));
}

template <typename K, typename A>
cudaError_t launch(K kern, dim3 grid, int smem, const A& a, cudaStream_t st) {
    if (smem >= 48 * 1024) {  // the prompts' kernel has static shared memory besides
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    kern<<<grid, kThreads, smem, st>>>(a);
    return cudaGetLastError();
}

// Channels a thread of the forward and the prompts: 16 bytes of x.
template <typename E> constexpr int kV = 16 / (int)sizeof(E);

}  // namespace conv

void conv_plan(ConvArgs& a, int io_bf16, bool backward) {
    const conv::Tile t = conv::tile_of(a.D, backward || !io_bf16 ? 4 : 8);
    a.cx = t.cx; a.ry = t.ry; a.nct = t.nct;
    a.G = conv::rows_per_piece(a.B, a.L, t, 0);
    a.nseg = a.L > 0 ? (a.L + a.G - 1) / a.G : 1;
    a.parts = (int)(((int64_t)a.B * a.nseg + t.ry - 1) / t.ry);
    a.Lq = ((size_t)a.L + 3) / 4 * 4;
}

cudaError_t launch_conv_fwd(const ConvArgs& a, int width, bool silu, int io_bf16, bool restore,
                            cudaStream_t st) {
    using namespace conv;
    const dim3 grid(a.parts, a.nct);
    return dispatch(width, silu, io_bf16, [&](auto e, auto w, auto s) {
        using E = typename decltype(e)::type;
        constexpr int W = decltype(w)::value, V = kV<E>;
        constexpr bool SL = decltype(s)::value != 0;
        if (restore)
            return launch(conv_fwd_kernel<E, V, W, SL, true, false>, grid, Fwd<E, V, W, SL, true, false>::kBytes, a, st);
        if (a.q_out)
            return launch(conv_fwd_kernel<E, V, W, SL, false, true>, grid, Fwd<E, V, W, SL, false, true>::kBytes, a, st);
        return launch(conv_fwd_kernel<E, V, W, SL, false, false>, grid, Fwd<E, V, W, SL, false, false>::kBytes, a, st);
    });
}

cudaError_t launch_conv_bwd(const ConvArgs& a, int width, bool silu, int io_bf16, cudaStream_t st) {
    using namespace conv;
    const dim3 grid(a.parts, a.nct);
    const cudaError_t e0 = dispatch(width, silu, io_bf16, [&](auto e, auto w, auto s) {
        using E = typename decltype(e)::type;
        constexpr int W = decltype(w)::value;
        constexpr bool SL = decltype(s)::value != 0;
        if (a.q) return launch(conv_bwd_kernel<E, W, SL, true>, grid, Bwd<E, true>::kBytes, a, st);
        return launch(conv_bwd_kernel<E, W, SL, false>, grid, Bwd<E, false>::kBytes, a, st);
    });
    if (e0 != cudaSuccess) return e0;
    conv_reduce_kernel<<<dim3((a.D + 31) / 32, width + 1), 256, 0, st>>>(a.part, a.parts, a.D, width, a.dw,
                                                                        a.dbias, a.status);
    return cudaGetLastError();
}

cudaError_t launch_conv_prompt(ConvServeArgs a, int width, bool silu, int io_bf16, cudaStream_t st) {
    using namespace conv;
    const Tile t = tile_of(a.D, io_bf16 ? 8 : 4);
    a.cx = t.cx; a.ry = t.ry;
    a.G = rows_per_piece(1, a.rows, t, a.S);
    a.items = (int64_t)(a.rows / a.G) + a.S;
    const dim3 grid((unsigned)((a.items + t.ry - 1) / t.ry), t.nct);
    return dispatch(width, silu, io_bf16, [&](auto e, auto w, auto s) {
        using E = typename decltype(e)::type;
        constexpr int W = decltype(w)::value, V = kV<E>;
        constexpr bool SL = decltype(s)::value != 0;
        return launch(conv_prompt_kernel<E, V, W, SL>, grid, Fwd<E, V, W, SL, false, false>::kBytes, a, st);
    });
}

cudaError_t launch_conv_step(const ConvServeArgs& a, int width, bool silu, int io_bf16, cudaStream_t st) {
    const int nvec = (a.D + 3) / 4;
    const int nt = nvec >= 256 ? 256 : (nvec + 31) / 32 * 32;
    const int tiles = (nvec + nt - 1) / nt;
    return conv::dispatch(width, silu, io_bf16, [&](auto e, auto w, auto s) {
        using E = typename decltype(e)::type;
        constexpr int W = decltype(w)::value;
        constexpr bool SL = decltype(s)::value != 0;
        // four rows a CTA once there are more rows than two CTAs an SM
        if ((int64_t)tiles * a.rows > 296)
            conv::conv_step_kernel<E, W, SL, 4><<<dim3(tiles, (a.rows + 3) / 4), nt, 0, st>>>(a);
        else
            conv::conv_step_kernel<E, W, SL, 1><<<dim3(tiles, a.rows), nt, 0, st>>>(a);
        return cudaGetLastError();
    });
}

}  // namespace ssm
