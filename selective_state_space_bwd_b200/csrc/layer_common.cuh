// Device helpers of the short convolution and of the serving calls: four-channel vectors, SiLU,
// and the lookup of the sequence that a work item of a packed batch belongs to.
#pragma once

#include "ssm_device.cuh"
#include "ssm_internal.h"

namespace ssm {

constexpr unsigned kFullWarp = 0xffffffffu;
constexpr unsigned kStatusInvalid = 1u;  // SSM_ERR_INVALID_ARG

// Records a condition when the caller gave a status word.
__device__ __forceinline__ void flag_if(unsigned* status, unsigned code) {
    if (status) flag_status(status, code);
}

// ---------------------------------------------------------------- V consecutive channels
// Raw vectors (as loaded) are kept apart from the conversion to V / 2 fp32 pairs.
__device__ __forceinline__ float2 bf16_pair(unsigned r) {
    return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
}
__device__ __forceinline__ unsigned pack_bf16(float2 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const unsigned*>(&a);
}
template <typename E, int V> struct Vec;
template <> struct Vec<float, 4> {
    using Raw = float4;
    static __device__ __forceinline__ Raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
    static __device__ __forceinline__ void unpack(const Raw& r, float2 (&o)[2]) {
        o[0] = make_float2(r.x, r.y);
        o[1] = make_float2(r.z, r.w);
    }
    static __device__ __forceinline__ Raw pack(const float2 (&v)[2]) {
        return make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    }
};
template <> struct Vec<__nv_bfloat16, 4> {
    using Raw = uint2;
    static __device__ __forceinline__ Raw zero() { return make_uint2(0u, 0u); }
    static __device__ __forceinline__ void unpack(const Raw& r, float2 (&o)[2]) {
        o[0] = bf16_pair(r.x);
        o[1] = bf16_pair(r.y);
    }
    static __device__ __forceinline__ Raw pack(const float2 (&v)[2]) {
        return make_uint2(pack_bf16(v[0]), pack_bf16(v[1]));
    }
};
template <> struct Vec<__nv_bfloat16, 8> {
    using Raw = uint4;
    static __device__ __forceinline__ Raw zero() { return make_uint4(0u, 0u, 0u, 0u); }
    static __device__ __forceinline__ void unpack(const Raw& r, float2 (&o)[4]) {
        o[0] = bf16_pair(r.x);
        o[1] = bf16_pair(r.y);
        o[2] = bf16_pair(r.z);
        o[3] = bf16_pair(r.w);
    }
    static __device__ __forceinline__ Raw pack(const float2 (&v)[4]) {
        return make_uint4(pack_bf16(v[0]), pack_bf16(v[1]), pack_bf16(v[2]), pack_bf16(v[3]));
    }
};
template <typename E, int V>
__device__ __forceinline__ typename Vec<E, V>::Raw ld_vec(const E* p) {
    return *reinterpret_cast<const typename Vec<E, V>::Raw*>(p);
}
template <typename E, int V>
__device__ __forceinline__ void st_vec(E* p, const float2 (&v)[V / 2]) {
    *reinterpret_cast<typename Vec<E, V>::Raw*>(p) = Vec<E, V>::pack(v);
}

// sigmoid(v) from the exp2 and reciprocal units.  exp(-v) overflows to infinity below -88, where the
// quotient is zero, as sigmoid is to fp32's normal numbers.  (One reciprocal for two quotients was
// tried: it saves one special-function operation in four but needs six instructions more a pair to
// keep infinities and NaN apart, and that unit is at most 59 % busy in these kernels: they wait for the fixed
// latency of dependent instructions.)
__device__ __forceinline__ float rcp_mufu(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 sigmoid_pair(float2 v) {
    const float2 z = __fmul2_rn(v, make_float2(-kLog2e, -kLog2e));
    const float2 a = __fadd2_rn(make_float2(ex2_mufu(z.x), ex2_mufu(z.y)), make_float2(1.f, 1.f));
    return make_float2(rcp_mufu(a.x), rcp_mufu(a.y));
}
__device__ __forceinline__ float2 silu_pair(float2 v) { return __fmul2_rn(v, sigmoid_pair(v)); }
__device__ __forceinline__ float silu_fast(float v) { return v * rcp_mufu(1.0f + ex2_mufu(-v * kLog2e)); }

// Row t (0..2^30) of an array whose rows lie ldb bytes apart (below 2^32): one 32 x 32 + 64 bit
// multiply-add.
template <typename T>
__device__ __forceinline__ T* row_at(T* base, int t, unsigned ldb) {
    return reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(base) + (unsigned long long)(unsigned)t * ldb);
}

// ---------------------------------------------------------------- packed sequences
// Time is cut into pieces of G rows that start at each sequence's first row.  Items number the
// pieces: sequence s owns items floor(offsets[s] / G) + s and up, which leaves room for its
// ceil(length / G) pieces and for one item where it is empty, since floor((o + l) / G) + 1 >=
// floor(o / G) + ceil(l / G); surplus items do nothing.  The whole batch then has
// floor(rows / G) + S items at most, whatever the lengths: no plan on the host, no pass over the
// offsets before the launch.
struct Span {
    int s;       // sequence
    int local;   // index of the piece within it
    int first;   // its first row, and the sequence's end
    int end;
    int slot;    // pool entry, or negative
    bool ok;     // the item has work: rows, or (local == 0) a state to write
};

__device__ __forceinline__ int64_t item_base(const int32_t* offsets, int s, int G) {
    return (int64_t)(offsets[s] / G) + s;
}

// The last sequence whose first item is at most `item`; the 32 lanes of a warp probe 32 places at
// a time, so 1024 sequences take two rounds of loads.
__device__ __forceinline__ int find_seq(const int32_t* offsets, int S, int G, int64_t item) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = S;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;
        const bool below = at < hi && item_base(offsets, at, G) <= item;
        const int n = __popc(__ballot_sync(kFullWarp, below));
        if (n == 0) break;  // the item lies before the first row
        lo += (n - 1) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

__device__ __forceinline__ int length_of(const int32_t* offsets, int s) {
    return (int)((unsigned)offsets[s + 1] - (unsigned)offsets[s]);
}

// Sequence s's rows, with everything that the device must not trust checked.  Does not look for
// repeated slots (see named_before).
__device__ __forceinline__ Span seq_span(const int32_t* offsets, const int32_t* slot, int s, int rows, int slots,
                                         int max_len) {
    Span r;
    const int o0 = offsets[s], o1 = offsets[s + 1];
    r.s = s;
    r.slot = slot[s];
    r.local = 0;
    r.first = o0;
    r.end = o1;
    r.ok = o0 >= 0 && o0 <= o1 && o1 <= rows && o1 - o0 <= max_len && r.slot < slots;
    return r;
}

// An item's rows: one piece of sequence s.
__device__ __forceinline__ Span item_span(const int32_t* offsets, const int32_t* slot, int s, int G,
                                          int64_t item, int rows, int slots) {
    Span r = seq_span(offsets, slot, s, rows, slots, rows);
    const int64_t local = item - item_base(offsets, s, G);
    r.ok = r.ok && local >= 0 && (local == 0 || local * G < r.end - r.first);
    r.local = r.ok ? (int)local : 0;
    r.first = r.ok ? r.first + r.local * G : 0;
    return r;
}

// Whether one of slot[0..s) equals slot[s] (a pool entry): the caller's share `t` of `nt`.
__device__ __forceinline__ bool named_before(const int32_t* slot, int s, int mine, int t, int nt) {
    bool hit = false;
    if (mine >= 0)
        for (int j = t; j < s; j += nt) hit |= slot[j] == mine;
    return hit;
}

// One CTA's look over the whole batch: offsets out of order or out of range, sequences that are
// too long, slots past the pool.
__device__ __forceinline__ void check_batch(const int32_t* offsets, const int32_t* slot, int S,
                                            int rows, int slots, int max_len, unsigned* status) {
    for (int s = threadIdx.x; s < S; s += blockDim.x) {
        const int o0 = offsets[s], o1 = offsets[s + 1];
        if (o0 < 0 || o1 < o0 || o1 > rows || o1 - o0 > max_len || slot[s] >= slots)
            flag_status(status, kStatusInvalid);
    }
}

}  // namespace ssm
