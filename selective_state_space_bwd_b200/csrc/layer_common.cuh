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

// ---------------------------------------------------------------- four consecutive channels
// Raw loads (16 bytes of fp32, 8 of bf16) are kept apart from the conversion so that several can
// be in flight.
template <typename E> struct Quad;
template <> struct Quad<float> {
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
template <> struct Quad<__nv_bfloat16> {
    using Raw = uint2;
    static __device__ __forceinline__ Raw zero() { return make_uint2(0u, 0u); }
    static __device__ __forceinline__ void unpack(const Raw& r, float2 (&o)[2]) {
        o[0] = make_float2(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u));
        o[1] = make_float2(__uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
    }
    static __device__ __forceinline__ Raw pack(const float2 (&v)[2]) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0].x, v[0].y);
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[1].x, v[1].y);
        return make_uint2(*reinterpret_cast<const unsigned*>(&a), *reinterpret_cast<const unsigned*>(&b));
    }
};
template <typename E>
__device__ __forceinline__ typename Quad<E>::Raw ld_quad(const E* p) {
    return *reinterpret_cast<const typename Quad<E>::Raw*>(p);
}
template <typename E>
__device__ __forceinline__ void st_quad(E* p, const float2 (&v)[2]) {
    *reinterpret_cast<typename Quad<E>::Raw*>(p) = Quad<E>::pack(v);
}

// v sigmoid(v).  exp(-v) overflows to infinity below -88, where the quotient is zero, as v sigmoid(v)
// is to fp32's smallest normal number.
__device__ __forceinline__ float silu_fast(float v) {
    return v * __fdividef(1.0f, 1.0f + ex2_mufu(-v * kLog2e));
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

// The item's rows, with everything that the device must not trust checked.  Does not look for
// repeated slots (see named_before).
__device__ __forceinline__ Span item_span(const int32_t* offsets, const int32_t* slot, int s, int G,
                                          int64_t item, int rows, int slots, int max_len) {
    Span r;
    r.s = s;
    const int o0 = offsets[s], o1 = offsets[s + 1];
    const int64_t local = item - item_base(offsets, s, G);
    r.slot = slot[s];
    r.end = o1;
    const bool sane = o0 >= 0 && o0 <= o1 && o1 <= rows && o1 - o0 <= max_len && r.slot < slots;
    r.ok = sane && local >= 0 && (local == 0 || local * G < o1 - o0);
    r.local = r.ok ? (int)local : 0;
    r.first = r.ok ? o0 + r.local * G : 0;
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
