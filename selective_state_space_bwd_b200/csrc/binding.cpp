// Python entry to the convolution and serving calls of libssm_scan.so (include/ssm_scan.h).
//
// Argument marshalling only, as the ctypes binding does it for the other calls: every tensor is checked
// (device, type, shape, strides), missing outputs are allocated on the current stream, and the C call is
// made on it.  It is compiled because these calls are short: a single token's kernels take 2 us, and
// reading ten tensors' attributes from Python takes five times that.
#include <torch/extension.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdint>
#include <optional>
#include <string>
#include <tuple>

#include "../../include/ssm_scan.h"

namespace {

namespace py = pybind11;
using at::Tensor;
using Opt = std::optional<Tensor>;

py::object& error_class() {
    static py::object* c = new py::object();  // outlives the interpreter's teardown
    return *c;
}

void check(int code, const char* what) {
    if (code == SSM_OK) return;
    PyErr_SetObject(error_class().ptr(), error_class()(code, what).ptr());
    throw py::error_already_set();
}

[[noreturn]] void refuse(const std::string& why) { throw py::value_error(why); }

std::string describe(const Tensor& t) {
    std::string s = std::string(c10::toString(t.scalar_type())) + " [";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + "] on " + t.device().str();
}

void expect_kind(const Tensor& t, const char* what, at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
    if (t.device() == dev && t.scalar_type() == type && t.sizes() == shape) return;
    std::string s;
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    refuse(std::string(what) + " must be " + c10::toString(type) + " [" + s + "] on " + dev.str() + ", is " +
           describe(t));
}

// A dense tensor of this shape, type and device; its address.
void* dense(const Tensor& t, const char* what, at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
    expect_kind(t, what, shape, type, dev);
    if (!t.is_contiguous()) refuse(std::string(what) + " must be contiguous");
    return t.data_ptr();
}
void* dense(const Opt& t, const char* what, at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
    return t ? dense(*t, what, shape, type, dev) : nullptr;
}

// A tensor of rows that may be strided: [..., D] with dense columns, its leading dimensions one row
// stride apart.  Its address, and the stride in elements (0: dense).
void* row_major(const Tensor& t, const char* what, at::IntArrayRef shape, at::ScalarType type, at::Device dev,
                int64_t& ld) {
    expect_kind(t, what, shape, type, dev);
    ld = 0;
    if (t.is_contiguous()) return t.data_ptr();
    int64_t rows = 1;
    for (int64_t i = t.dim() - 2; i >= 0; --i) {
        if (t.size(i) == 1) continue;
        if (rows == 1)
            ld = t.stride(i);
        else if (t.stride(i) != ld * rows)
            refuse(std::string(what) + ": rows must lie one stride apart");
        rows *= t.size(i);
    }
    if (t.stride(-1) != 1 || (rows > 1 && ld < t.size(-1)))
        refuse(std::string(what) + ": columns must be dense and rows must not overlap");
    return t.data_ptr();
}
void* row_major(const Opt& t, const char* what, at::IntArrayRef shape, at::ScalarType type, at::Device dev,
                int64_t& ld) {
    ld = 0;
    return t ? row_major(*t, what, shape, type, dev, ld) : nullptr;
}

int32_t io_of(at::ScalarType t) {
    if (t == at::kFloat) return SSM_F32;
    if (t == at::kBFloat16) return SSM_BF16;
    refuse(std::string("unsupported io dtype ") + c10::toString(t));
}

// Device and element type of a call, from its first tensor.
struct Call {
    at::Device dev;
    at::ScalarType type;
    int32_t io;
    c10::cuda::CUDAGuard guard;
    Call(const Tensor& t, const char* what, int64_t ndim)
        : dev(t.device()), type(t.scalar_type()), io(check_first(t, what, ndim)), guard(t.device()) {}
    static int32_t check_first(const Tensor& t, const char* what, int64_t ndim) {
        if (!t.is_cuda() || t.dim() != ndim)
            refuse(std::string(what) + " must be a CUDA tensor of " + std::to_string(ndim) + " dimensions");
        return io_of(t.scalar_type());
    }
    ssm_stream_t stream() const {
        return reinterpret_cast<ssm_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
    }
    Tensor empty(at::IntArrayRef shape, at::ScalarType t) const {
        return at::empty(shape, at::TensorOptions().dtype(t).device(dev));
    }
};

int64_t taps(const Tensor& w, const Opt& bias, int64_t D, const Call& c, const float*& pw, const float*& pb) {
    if (w.dim() != 2) refuse("w must be [D, W]");
    pw = static_cast<const float*>(dense(w, "w", {D, w.size(1)}, at::kFloat, c.dev));
    pb = static_cast<const float*>(dense(bias, "bias", {D}, at::kFloat, c.dev));
    return w.size(1);
}

void* workspace(const Opt& ws, const Call& c, size_t& bytes) {
    bytes = 0;
    if (!ws) return nullptr;
    if (ws->device() != c.dev || !ws->is_contiguous()) refuse("ws must be a contiguous tensor on " + c.dev.str());
    bytes = ws->nbytes();
    return ws->data_ptr();
}

void q8_of(const Opt& q, const Opt& qe, int64_t B, int64_t L, int64_t D, const Call& c, int8_t*& pq, uint8_t*& pe) {
    pq = static_cast<int8_t*>(dense(q, "q", {B, L, D}, at::kChar, c.dev));
    pe = static_cast<uint8_t*>(dense(qe, "qe", {B, (D + 31) / 32, (L + 3) / 4 * 4}, at::kByte, c.dev));
}

// ---------------------------------------------------------------- convolution
std::tuple<Tensor, Opt, Opt, Opt> conv_fwd(const Tensor& x, const Tensor& w, const Opt& bias, bool silu, const Opt& s0,
                                           bool want_sL, bool want_q8, Opt y, Opt sL, Opt q, Opt qe) {
    const Call c(x, "x", 3);
    const int64_t B = x.size(0), L = x.size(1), D = x.size(2);
    ssm_conv_shape s = {};
    const float *pw, *pb;
    const int64_t W = taps(w, bias, D, c, pw, pb);
    s.batch = B; s.seqlen = L; s.dim = D; s.width = (int32_t)W; s.io = c.io; s.flags = silu ? SSM_CONV_SILU : 0;
    if (!y) y = c.empty({B, L, D}, c.type);
    if (!sL && want_sL) sL = c.empty({B, W - 1, D}, c.type);
    if (!q && want_q8) {
        q = c.empty({B, L, D}, at::kChar);
        qe = c.empty({B, (D + 31) / 32, (L + 3) / 4 * 4}, at::kByte);
    }
    int8_t* pq;
    uint8_t* pe;
    q8_of(q, qe, B, L, D, c, pq, pe);
    const void* px = row_major(x, "x", x.sizes(), c.type, c.dev, s.ldx);
    void* py = row_major(*y, "y", x.sizes(), c.type, c.dev, s.ldy);
    const void* p0 = dense(s0, "s0", {B, W - 1, D}, c.type, c.dev);
    void* pl = dense(sL, "sL", {B, W - 1, D}, c.type, c.dev);
    check(ssm_conv_fwd(&s, px, pw, pb, p0, py, pl, pq, pe, c.stream()), "ssm_conv_fwd");
    return {*y, sL, q, qe};
}

Tensor conv_restore(const Tensor& q, const Tensor& qe, const Tensor& w, const Opt& bias, bool silu, const Opt& s0,
                    at::ScalarType type, Opt y) {
    if (!q.is_cuda() || q.dim() != 3) refuse("q must be a CUDA tensor [B, L, D]");
    const int64_t B = q.size(0), L = q.size(1), D = q.size(2);
    c10::cuda::CUDAGuard guard(q.device());
    if (!y) y = at::empty({B, L, D}, at::TensorOptions().dtype(type).device(q.device()));
    const Call c(*y, "y", 3);
    ssm_conv_shape s = {};
    const float *pw, *pb;
    const int64_t W = taps(w, bias, D, c, pw, pb);
    s.batch = B; s.seqlen = L; s.dim = D; s.width = (int32_t)W; s.io = c.io; s.flags = silu ? SSM_CONV_SILU : 0;
    int8_t* pq;
    uint8_t* pe;
    q8_of(q, qe, B, L, D, c, pq, pe);
    void* py = row_major(*y, "y", {B, L, D}, type, q.device(), s.ldy);
    const void* p0 = dense(s0, "s0", {B, W - 1, D}, type, c.dev);
    check(ssm_conv_restore(&s, pq, pe, pw, pb, p0, py, c.stream()), "ssm_conv_restore");
    return *y;
}

std::tuple<Tensor, Tensor, Opt, Opt> conv_bwd(const Opt& x, const Opt& q, const Opt& qe, const Tensor& w,
                                              const Opt& bias, const Tensor& dy, bool silu, const Opt& s0,
                                              const Opt& dsL, bool want_ds0, Opt dx, Opt dw, Opt dbias, Opt ds0,
                                              const Opt& ws) {
    const Call c(dy, "dy", 3);
    if (x.has_value() == q.has_value()) refuse("give either x or q8");
    const int64_t B = dy.size(0), L = dy.size(1), D = dy.size(2);
    ssm_conv_shape s = {};
    const float *pw, *pb;
    const int64_t W = taps(w, bias, D, c, pw, pb);
    s.batch = B; s.seqlen = L; s.dim = D; s.width = (int32_t)W; s.io = c.io; s.flags = silu ? SSM_CONV_SILU : 0;
    if (!dx) dx = c.empty({B, L, D}, c.type);
    if (!dw) dw = c.empty({D, W}, at::kFloat);
    if (!dbias && bias) dbias = c.empty({D}, at::kFloat);
    if (!ds0 && want_ds0) ds0 = c.empty({B, W - 1, D}, c.type);
    const void* px = row_major(x, "x", dy.sizes(), c.type, c.dev, s.ldx);
    int8_t* pq;
    uint8_t* pe;
    q8_of(q, qe, B, L, D, c, pq, pe);
    const void* pg = row_major(dy, "dy", dy.sizes(), c.type, c.dev, s.lddy);
    void* pdx = row_major(*dx, "dx", dy.sizes(), c.type, c.dev, s.lddx);
    const void* p0 = dense(s0, "s0", {B, W - 1, D}, c.type, c.dev);
    const void* pl = dense(dsL, "dsL", {B, W - 1, D}, c.type, c.dev);
    float* pdw = static_cast<float*>(dense(*dw, "dw", {D, W}, at::kFloat, c.dev));
    float* pdb = static_cast<float*>(dense(dbias, "dbias", {D}, at::kFloat, c.dev));
    void* pd0 = dense(ds0, "ds0", {B, W - 1, D}, c.type, c.dev);
    size_t n;
    void* pws = workspace(ws, c, n);
    Tensor own;
    if (!pws) {  // freed on return: its memory is only handed out again in this stream's order
        n = ssm_conv_workspace_bytes(&s);
        own = c.empty({(int64_t)(n > 256 ? n : 256)}, at::kByte);
        pws = own.data_ptr();
    }
    check(ssm_conv_bwd(&s, px, pq, pe, pw, pb, p0, pg, pl, pdx, pdw, pdb, pd0, pws, n, c.stream()), "ssm_conv_bwd");
    return {*dx, *dw, dbias, ds0};
}

// ---------------------------------------------------------------- serving
// offsets, slots and carry of a packed batch, or slots alone
struct Index {
    int64_t seqs = 0;
    const int32_t* offsets = nullptr;
    const int32_t* slot = nullptr;
    const uint8_t* carry = nullptr;
    Index(const Opt& off, const Opt& slots, const Opt& cry, int64_t rows, const Call& c) {
        if (!off) {
            slot = static_cast<const int32_t*>(dense(slots, "slots", {rows}, at::kInt, c.dev));
            return;
        }
        if (off->dim() != 1 || off->size(0) < 1) refuse("offsets must hold one int32 a sequence and one more");
        if (!slots) refuse("slots is needed");
        seqs = off->size(0) - 1;
        offsets = static_cast<const int32_t*>(dense(*off, "offsets", {seqs + 1}, at::kInt, c.dev));
        slot = static_cast<const int32_t*>(dense(*slots, "slots", {seqs}, at::kInt, c.dev));
        if (cry)
            carry = static_cast<const uint8_t*>(
                dense(*cry, "carry", {seqs}, cry->scalar_type() == at::kBool ? at::kBool : at::kByte, c.dev));
    }
};

Tensor conv_serve(const Tensor& x, const Tensor& w, const Opt& bias, const Opt& offsets, const Opt& slots,
                  const Tensor& pool, const Opt& carry, bool silu, Opt y, const Opt& ws) {
    const Call c(x, "x", 2);
    const int64_t R = x.size(0), D = x.size(1);
    ssm_conv_serve s = {};
    const float *pw, *pb;
    const int64_t W = taps(w, bias, D, c, pw, pb);
    if (pool.dim() != 3) refuse("pool must be [slots, W-1, D]");
    void* pp = dense(pool, "pool", {pool.size(0), W - 1, D}, c.type, c.dev);
    const Index ix(offsets, slots, carry, R, c);
    size_t n;
    void* pws = workspace(ws, c, n);
    if (!y) y = c.empty({R, D}, c.type);
    s.rows = R; s.seqs = ix.seqs; s.dim = D; s.slots = pool.size(0);
    s.width = (int32_t)W; s.io = c.io; s.flags = silu ? SSM_CONV_SILU : 0;
    const void* px = row_major(x, "x", x.sizes(), c.type, c.dev, s.ldx);
    void* py = row_major(*y, "y", x.sizes(), c.type, c.dev, s.ldy);
    if (offsets)
        check(ssm_conv_prompt(&s, px, pw, pb, ix.offsets, ix.slot, ix.carry, pp, py, pws, n, c.stream()),
              "ssm_conv_prompt");
    else
        check(ssm_conv_step(&s, px, pw, pb, ix.slot, pp, py, pws, n, c.stream()), "ssm_conv_step");
    return *y;
}

Tensor scan_serve(const Tensor& x, const Tensor& delta_raw, const Tensor& A_log, const Tensor& Bm, const Tensor& Cm,
                  const Tensor& Dskip, const Opt& offsets, const Opt& slots, const Tensor& pool, const Opt& carry,
                  const Opt& z, bool zoh, int64_t max_len, Opt y, const Opt& ws) {
    const Call c(x, "x", 2);
    const int64_t R = x.size(0), D = x.size(1);
    if (A_log.dim() != 2) refuse("A_log must be [D, N]");
    const int64_t N = A_log.size(1);
    ssm_scan_serve s = {};
    const float* pa = static_cast<const float*>(dense(A_log, "A_log", {D, N}, at::kFloat, c.dev));
    const float* pd = static_cast<const float*>(dense(Dskip, "Dskip", {D}, at::kFloat, c.dev));
    if (pool.dim() != 3) refuse("pool must be [slots, D, N]");
    float* pp = static_cast<float*>(dense(pool, "pool", {pool.size(0), D, N}, at::kFloat, c.dev));
    const Index ix(offsets, slots, carry, R, c);
    size_t n;
    void* pws = workspace(ws, c, n);
    if (!y) y = c.empty({R, D}, c.type);
    s.rows = R; s.seqs = ix.seqs; s.dim = D; s.dstate = N; s.slots = pool.size(0); s.max_len = max_len;
    s.io = c.io; s.discretization = zoh ? SSM_ZOH : SSM_EULER;
    const void* px = row_major(x, "x", x.sizes(), c.type, c.dev, s.ldx);
    const void* pr = row_major(delta_raw, "delta_raw", x.sizes(), c.type, c.dev, s.lddelta);
    const void* pz = row_major(z, "z", x.sizes(), c.type, c.dev, s.ldz);
    const void* pB = row_major(Bm, "Bm", {R, N}, c.type, c.dev, s.ldb);
    const void* pC = row_major(Cm, "Cm", {R, N}, c.type, c.dev, s.ldc);
    void* py = row_major(*y, "y", x.sizes(), c.type, c.dev, s.ldy);
    if (offsets)
        check(ssm_scan_prompt(&s, px, pr, pa, pB, pC, pd, pz, ix.offsets, ix.slot, ix.carry, pp, py, pws, n, c.stream()),
              "ssm_scan_prompt");
    else
        check(ssm_scan_step(&s, px, pr, pa, pB, pC, pd, pz, ix.slot, pp, py, pws, n, c.stream()), "ssm_scan_step");
    return *y;
}

}  // namespace

PYBIND11_MODULE(_ssm_torch, m) {
    m.attr("built_against") = SSM_BUILT_AGAINST;  // compared before the first call
    m.def("set_error_class", [](py::object c) { error_class() = std::move(c); });
    m.def("conv_fwd", &conv_fwd);
    m.def("conv_restore", &conv_restore);
    m.def("conv_bwd", &conv_bwd);
    m.def("conv_serve", &conv_serve);
    m.def("scan_serve", &scan_serve);
}
