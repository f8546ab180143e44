// C-ABI entry points of the short convolution and of the serving calls (include/ssm_scan.h):
// argument validation on the host, workspace layout, kernel launches.  Nothing here allocates
// memory or keeps state between calls.
#include "../../include/ssm_scan.h"
#include "api_util.h"
#include "ssm_internal.h"

#include <cuda_runtime.h>
#include <stdint.h>

using namespace ssm_api;

namespace {

int check_io(int32_t io) { return io == SSM_F32 || io == SSM_BF16 ? SSM_OK : SSM_ERR_UNSUPPORTED; }

// A row stride (0 = the row's length): at least the row, a multiple of `unit` elements, and below 2^29, so
// that its bytes fit 32 bits.
int check_ld(int64_t ld, int64_t len, int64_t unit) {
    if (ld == 0) return SSM_OK;
    if (ld < len) return SSM_ERR_INVALID_ARG;
    if (ld > (int64_t)1 << 29) return SSM_ERR_UNSUPPORTED;
    return ld % unit == 0 ? SSM_OK : SSM_ERR_MISALIGNED;
}
size_t stride(int64_t ld, int64_t len) { return (size_t)(ld ? ld : len); }

bool aligned_to(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

int esize(int32_t io) { return io == SSM_BF16 ? 2 : 4; }

int check_conv(const ssm_conv_shape* s) {
    if (!s) return SSM_ERR_INVALID_ARG;
    if (s->batch < 0 || s->seqlen < 0 || s->dim < 1 || s->reserved != 0) return SSM_ERR_INVALID_ARG;
    if ((s->flags & ~SSM_CONV_SILU) != 0) return SSM_ERR_INVALID_ARG;
    if (check_io(s->io) != SSM_OK || s->width < 2 || s->width > 4) return SSM_ERR_UNSUPPORTED;
    if (s->batch > 65535 || s->seqlen > (int64_t)1 << 30 || s->dim > (int64_t)1 << 22 ||
        s->batch * s->seqlen > (int64_t)1 << 34)
        return SSM_ERR_UNSUPPORTED;
    const int64_t unit = 16 / esize(s->io);
    if (s->dim % unit != 0) return SSM_ERR_MISALIGNED;
    for (int64_t ld : {s->ldx, s->ldy, s->lddy, s->lddx})
        if (int st = check_ld(ld, s->dim, unit)) return st;
    return SSM_OK;
}

ssm::ConvArgs conv_args(const ssm_conv_shape* s, bool backward) {
    ssm::ConvArgs a = {};
    a.B = (int)s->batch; a.L = (int)s->seqlen; a.D = (int)s->dim;
    a.ldx = stride(s->ldx, s->dim); a.ldy = stride(s->ldy, s->dim);
    a.lddy = stride(s->lddy, s->dim); a.lddx = stride(s->lddx, s->dim);
    ssm::conv_plan(a, s->io == SSM_BF16, backward);
    return a;
}

size_t conv_part_bytes(const ssm::ConvArgs& a, int width) {
    return (size_t)a.parts * (width + 1) * a.D * sizeof(float);
}

int launch_status(cudaError_t e) { return e == cudaSuccess ? SSM_OK : SSM_ERR_CUDA; }

// The status word of a call whose workspace may be absent: *status is null without one.
int find_status(void* ws, size_t ws_bytes, unsigned** status) {
    *status = nullptr;
    if (!ws) return ws_bytes ? SSM_ERR_INVALID_ARG : SSM_OK;
    if (!aligned16(ws)) return SSM_ERR_MISALIGNED;
    if (ws_bytes < kStatusBytes) return SSM_ERR_WORKSPACE_TOO_SMALL;
    *status = at<unsigned>(ws, 0);
    return SSM_OK;
}

int clear_status(unsigned* status, cudaStream_t s) {
    if (!status) return SSM_OK;
    return launch_status(cudaMemsetAsync(status, 0, sizeof(unsigned), s));
}

// offsets, slot and carry of a packed batch (prompts) or slot alone (single tokens)
int check_index(const int32_t* offsets, const int32_t* slot, bool prompts) {
    if (prompts && (!offsets || !slot)) return SSM_ERR_INVALID_ARG;
    if (!aligned_to(offsets, 4) || !aligned_to(slot, 4)) return SSM_ERR_MISALIGNED;
    return SSM_OK;
}

// Sequences or rows that may name pool entries: each is compared with all before it by every CTA that
// works on it.  4096 single tokens of 4096 channels with 16 states take 64 tiles of channels a row, 2.1 GB of cached
// loads: 475 us, against 358 without slots, which need no comparison.
constexpr int64_t kMaxNamed = 4096;

int check_rows(int64_t rows, int64_t seqs, int64_t slots, bool prompts) {
    if (rows < 0 || seqs < 0 || slots < 0) return SSM_ERR_INVALID_ARG;
    if (!prompts && seqs != 0) return SSM_ERR_INVALID_ARG;
    if (rows > (int64_t)1 << 30 || seqs > kMaxNamed || slots > (int64_t)1 << 30) return SSM_ERR_UNSUPPORTED;
    if (!prompts && rows > 65535) return SSM_ERR_UNSUPPORTED;
    return SSM_OK;
}

int check_conv_serve(const ssm_conv_serve* s, bool prompts) {
    if (!s) return SSM_ERR_INVALID_ARG;
    if (s->dim < 1 || s->reserved != 0 || (s->flags & ~SSM_CONV_SILU) != 0) return SSM_ERR_INVALID_ARG;
    if (int st = check_rows(s->rows, s->seqs, s->slots, prompts)) return st;
    if (check_io(s->io) != SSM_OK || s->width < 2 || s->width > 4 || s->dim > (int64_t)1 << 22)
        return SSM_ERR_UNSUPPORTED;
    const int64_t unit = 16 / esize(s->io);
    if (s->dim % unit != 0) return SSM_ERR_MISALIGNED;
    for (int64_t ld : {s->ldx, s->ldy})
        if (int st = check_ld(ld, s->dim, unit)) return st;
    return SSM_OK;
}

int conv_serve(const ssm_conv_serve* s, bool prompts, const void* x, const float* w,
               const float* bias, const int32_t* offsets, const int32_t* slot, const uint8_t* carry,
               void* pool, void* y, void* ws, size_t ws_bytes, ssm_stream_t stream) {
    int st = check_conv_serve(s, prompts);
    if (st != SSM_OK) return st;
    const size_t rows = s->rows, D = s->dim;
    const void* ptrs[] = {x, w, bias, pool, y};
    const size_t counts[] = {rows, D, bias ? D : 0, (size_t)s->slots, rows};
    if ((st = check_arrays(ptrs, counts, 5)) != SSM_OK) return st;
    if (rows && x == y) return SSM_ERR_INVALID_ARG;
    const bool work = prompts ? s->seqs > 0 : rows > 0;
    if (work && (st = check_index(offsets, slot, prompts)) != SSM_OK) return st;
    if (!prompts && !slot && s->rows > s->slots) return SSM_ERR_INVALID_ARG;
    if (!prompts && slot && s->rows > kMaxNamed) return SSM_ERR_UNSUPPORTED;
    ssm::ConvServeArgs a = {};
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if ((st = find_status(ws, ws_bytes, &a.status)) != SSM_OK) return st;
    if ((st = clear_status(a.status, cs)) != SSM_OK || !work) return st;
    a.rows = (int)rows; a.S = (int)s->seqs; a.D = (int)D; a.slots = (int)s->slots;
    a.ldx = stride(s->ldx, s->dim); a.ldy = stride(s->ldy, s->dim);
    a.x = x; a.w = w; a.bias = bias; a.offsets = offsets; a.slot = slot; a.carry = carry;
    a.pool = pool; a.y = y;
    const bool silu = (s->flags & SSM_CONV_SILU) != 0;
    return launch_status(prompts ? ssm::launch_conv_prompt(a, s->width, silu, s->io == SSM_BF16, cs)
                                 : ssm::launch_conv_step(a, s->width, silu, s->io == SSM_BF16, cs));
}

int check_scan_serve(const ssm_scan_serve* s, bool prompts) {
    if (!s) return SSM_ERR_INVALID_ARG;
    if (s->dim < 1 || s->max_len < 0 || (!prompts && s->max_len != 0)) return SSM_ERR_INVALID_ARG;
    if (s->discretization != SSM_EULER && s->discretization != SSM_ZOH) return SSM_ERR_INVALID_ARG;
    if (int st = check_rows(s->rows, s->seqs, s->slots, prompts)) return st;
    if (check_io(s->io) != SSM_OK || s->dim > (int64_t)1 << 20) return SSM_ERR_UNSUPPORTED;
    if (s->dstate != 4 && s->dstate != 8 && s->dstate != 16) return SSM_ERR_UNSUPPORTED;
    const int64_t tile = 256 / s->dstate;  // channels of a prompt CTA: the grid holds 2^31 - 1 CTAs
    if (s->seqs * ((s->dim + tile - 1) / tile) > (int64_t)0x7fffffff) return SSM_ERR_UNSUPPORTED;
    const int64_t unit = 16 / esize(s->io);
    if (s->dim % unit != 0) return SSM_ERR_MISALIGNED;
    for (int64_t ld : {s->ldx, s->lddelta, s->ldz, s->ldy})
        if (int st = check_ld(ld, s->dim, unit)) return st;
    for (int64_t ld : {s->ldb, s->ldc})
        if (int st = check_ld(ld, s->dstate, 4)) return st;
    return SSM_OK;
}

int scan_serve(const ssm_scan_serve* s, bool prompts, const void* x, const void* delta_raw,
               const float* A_log, const void* Bm, const void* Cm, const float* Dskip, const void* z,
               const int32_t* offsets, const int32_t* slot, const uint8_t* carry, float* pool,
               void* y, void* ws, size_t ws_bytes, ssm_stream_t stream) {
    int st = check_scan_serve(s, prompts);
    if (st != SSM_OK) return st;
    const size_t rows = s->rows, D = s->dim, N = s->dstate;
    const void* ptrs[] = {x, delta_raw, z, A_log, Dskip, pool, y};
    const size_t counts[] = {rows, rows, z ? rows : 0, D * N, D, (size_t)s->slots, rows};
    if ((st = check_arrays(ptrs, counts, 7)) != SSM_OK) return st;
    for (const void* p : {Bm, Cm}) {
        if (!ptr_ok(p, rows)) return SSM_ERR_INVALID_ARG;
        if (rows && !aligned_to(p, 4 * esize(s->io))) return SSM_ERR_MISALIGNED;
    }
    if (rows && (y == x || y == delta_raw || y == z)) return SSM_ERR_INVALID_ARG;
    const bool work = prompts ? s->seqs > 0 : rows > 0;
    if (work && (st = check_index(offsets, slot, prompts)) != SSM_OK) return st;
    if (!prompts && !slot && s->rows > s->slots) return SSM_ERR_INVALID_ARG;
    if (!prompts && slot && s->rows > kMaxNamed) return SSM_ERR_UNSUPPORTED;
    ssm::ScanServeArgs a = {};
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if ((st = find_status(ws, ws_bytes, &a.status)) != SSM_OK) return st;
    if ((st = clear_status(a.status, cs)) != SSM_OK || !work) return st;
    a.rows = (int)rows; a.S = (int)s->seqs; a.D = (int)D; a.slots = (int)s->slots;
    a.max_len = s->max_len && s->max_len < s->rows ? (int)s->max_len : (int)rows;
    a.zoh = s->discretization == SSM_ZOH;
    a.ldx = stride(s->ldx, s->dim); a.ldd = stride(s->lddelta, s->dim);
    a.ldz = stride(s->ldz, s->dim); a.ldy = stride(s->ldy, s->dim);
    a.ldb = stride(s->ldb, s->dstate); a.ldc = stride(s->ldc, s->dstate);
    a.x = x; a.draw = delta_raw; a.A_log = A_log; a.Bm = Bm; a.Cm = Cm; a.Dskip = Dskip; a.z = z;
    a.offsets = offsets; a.slot = slot; a.carry = carry; a.pool = pool; a.y = y;
    return launch_status(prompts ? ssm::launch_scan_prompt(a, s->io == SSM_BF16, (int)N, cs)
                                 : ssm::launch_scan_step(a, s->io == SSM_BF16, (int)N, cs));
}

}  // namespace

extern "C" {

size_t ssm_conv_workspace_bytes(const ssm_conv_shape* shape) {
    if (check_conv(shape) != SSM_OK) return 0;
    return kStatusBytes + align256(conv_part_bytes(conv_args(shape, true), shape->width));
}

int ssm_conv_fwd(const ssm_conv_shape* shape, const void* x, const float* w, const float* bias,
                 const void* s0, void* y, void* sL, int8_t* q, uint8_t* qe, ssm_stream_t stream) {
    int st = check_conv(shape);
    if (st != SSM_OK) return st;
    const size_t B = shape->batch, M = B * shape->seqlen, D = shape->dim;
    if ((q == nullptr) != (qe == nullptr) && M) return SSM_ERR_INVALID_ARG;
    const void* ptrs[] = {x, w, bias, s0, y, sL, q, qe};
    const size_t counts[] = {M, D, bias ? D : 0, s0 ? B : 0, M, sL ? B : 0, q ? M : 0, q ? M : 0};
    if ((st = check_arrays(ptrs, counts, 8)) != SSM_OK) return st;
    if ((M && x == y) || (sL && sL == s0)) return SSM_ERR_INVALID_ARG;
    if (B == 0 || (M == 0 && !sL)) return SSM_OK;
    ssm::ConvArgs a = conv_args(shape, false);
    a.x = x; a.w = w; a.bias = bias; a.s0 = s0; a.y = y; a.sL = sL; a.q_out = q; a.qe_out = qe;
    return launch_status(ssm::launch_conv_fwd(a, shape->width, (shape->flags & SSM_CONV_SILU) != 0,
                                              shape->io == SSM_BF16, false,
                                              reinterpret_cast<cudaStream_t>(stream)));
}

int ssm_conv_restore(const ssm_conv_shape* shape, const int8_t* q, const uint8_t* qe,
                     const float* w, const float* bias, const void* s0, void* y,
                     ssm_stream_t stream) {
    int st = check_conv(shape);
    if (st != SSM_OK) return st;
    const size_t B = shape->batch, M = B * shape->seqlen, D = shape->dim;
    const void* ptrs[] = {q, qe, w, bias, s0, y};
    const size_t counts[] = {M, M, D, bias ? D : 0, s0 ? B : 0, M};
    if ((st = check_arrays(ptrs, counts, 6)) != SSM_OK) return st;
    if (M == 0) return SSM_OK;
    ssm::ConvArgs a = conv_args(shape, false);
    a.q = q; a.qe = qe; a.w = w; a.bias = bias; a.s0 = s0; a.y = y;
    return launch_status(ssm::launch_conv_fwd(a, shape->width, (shape->flags & SSM_CONV_SILU) != 0,
                                              shape->io == SSM_BF16, true,
                                              reinterpret_cast<cudaStream_t>(stream)));
}

int ssm_conv_bwd(const ssm_conv_shape* shape, const void* x, const int8_t* q, const uint8_t* qe,
                 const float* w, const float* bias, const void* s0, const void* dy,
                 const void* dsL, void* dx, float* dw, float* dbias, void* ds0, void* ws,
                 size_t ws_bytes, ssm_stream_t stream) {
    int st = check_conv(shape);
    if (st != SSM_OK) return st;
    const size_t B = shape->batch, M = B * shape->seqlen, D = shape->dim, W = shape->width;
    // exactly one source of the input
    if (M && (x ? q || qe : !q || !qe)) return SSM_ERR_INVALID_ARG;
    const void* ptrs[] = {x, q, qe, w, bias, s0, dy, dsL, dx, dw, dbias, ds0, ws};
    const size_t counts[] = {x ? M : 0, q ? M : 0, qe ? M : 0, D, bias ? D : 0, s0 ? B : 0, M,
                             dsL ? B : 0, M, D, dbias ? D : 0, ds0 ? B : 0, 1};
    if ((st = check_arrays(ptrs, counts, 13)) != SSM_OK) return st;
    if (M && (dx == x || dx == dy)) return SSM_ERR_INVALID_ARG;
    if (ds0 && (ds0 == s0 || ds0 == dsL)) return SSM_ERR_INVALID_ARG;
    if (ws_bytes < ssm_conv_workspace_bytes(shape)) return SSM_ERR_WORKSPACE_TOO_SMALL;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (M == 0) {  // no steps: the state passes through, the sums are empty
        if (cudaMemsetAsync(ws, 0, sizeof(unsigned), s) != cudaSuccess) return SSM_ERR_CUDA;
        if (cudaMemsetAsync(dw, 0, D * W * sizeof(float), s) != cudaSuccess) return SSM_ERR_CUDA;
        if (dbias && cudaMemsetAsync(dbias, 0, D * sizeof(float), s) != cudaSuccess) return SSM_ERR_CUDA;
        const size_t n = ds0 ? B * (W - 1) * D * esize(shape->io) : 0;
        if (n == 0) return SSM_OK;
        return launch_status(dsL ? cudaMemcpyAsync(ds0, dsL, n, cudaMemcpyDeviceToDevice, s)
                                 : cudaMemsetAsync(ds0, 0, n, s));
    }
    ssm::ConvArgs a = conv_args(shape, true);
    a.x = x; a.q = q; a.qe = qe; a.w = w; a.bias = bias; a.s0 = s0; a.dy = dy; a.dsL = dsL;
    a.dx = dx; a.dw = dw; a.dbias = dbias; a.ds0 = ds0;
    a.status = at<unsigned>(ws, 0);
    a.part = at<float>(ws, kStatusBytes);
    return launch_status(ssm::launch_conv_bwd(a, shape->width, (shape->flags & SSM_CONV_SILU) != 0,
                                              shape->io == SSM_BF16, s));
}

int ssm_conv_prompt(const ssm_conv_serve* shape, const void* x, const float* w, const float* bias,
                    const int32_t* offsets, const int32_t* slot, const uint8_t* carry, void* pool,
                    void* y, void* ws, size_t ws_bytes, ssm_stream_t stream) {
    return conv_serve(shape, true, x, w, bias, offsets, slot, carry, pool, y, ws, ws_bytes, stream);
}

int ssm_conv_step(const ssm_conv_serve* shape, const void* x, const float* w, const float* bias,
                  const int32_t* slot, void* pool, void* y, void* ws, size_t ws_bytes,
                  ssm_stream_t stream) {
    return conv_serve(shape, false, x, w, bias, nullptr, slot, nullptr, pool, y, ws, ws_bytes, stream);
}

int ssm_scan_prompt(const ssm_scan_serve* shape, const void* x, const void* delta_raw,
                    const float* A_log, const void* Bm, const void* Cm, const float* Dskip,
                    const void* z, const int32_t* offsets, const int32_t* slot,
                    const uint8_t* carry, float* pool, void* y, void* ws, size_t ws_bytes,
                    ssm_stream_t stream) {
    return scan_serve(shape, true, x, delta_raw, A_log, Bm, Cm, Dskip, z, offsets, slot, carry,
                      pool, y, ws, ws_bytes, stream);
}

int ssm_scan_step(const ssm_scan_serve* shape, const void* x, const void* delta_raw,
                  const float* A_log, const void* Bm, const void* Cm, const float* Dskip,
                  const void* z, const int32_t* slot, float* pool, void* y, void* ws,
                  size_t ws_bytes, ssm_stream_t stream) {
    return scan_serve(shape, false, x, delta_raw, A_log, Bm, Cm, Dskip, z, nullptr, slot, nullptr,
                      pool, y, ws, ws_bytes, stream);
}

}  // extern "C"
