// binding.cpp -- argument marshalling of the calls that may be a few microseconds
// of work on the device (gated recurrence, layer norm, cross entropy, AdamW): the
// checks, the outputs and the C ABI call of each in one native function, where the
// same in Python took several times the launch itself (measured on the Grace host:
// glr_bwd 48 us, an AdamW step over 90 tensors 350 us).  No step of any operation is
// here.  Argument errors raise ValueError (TypeError for a storage type that is
// neither float32 nor bfloat16), library statuses go to the package's _check.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <pybind11/pybind11.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>
#include <vector>

#include "lrscan.h"

namespace py = pybind11;

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

// A tensor argument; None is an undefined tensor.
Tensor arg(const char* name, const py::object& o) {
    if (o.is_none()) return Tensor();
    if (!THPVariable_Check(o.ptr())) throw py::type_error(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o.ptr());
}
Tensor need(const char* name, const py::object& o) {
    Tensor t = arg(name, o);
    if (!t.defined()) throw py::type_error(std::string(name) + " must be a tensor, not None");
    return t;
}
py::object wrap(const Tensor& t) {
    if (!t.defined()) return py::none();
    return py::reinterpret_steal<py::object>(THPVariable_Wrap(t));
}

std::string text(const Tensor& t) {
    std::string s = std::string(c10::toString(t.scalar_type())) + " [";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + "] on " + t.device().str() + (t.is_contiguous() ? "" : ", not contiguous");
}
std::string text(IntArrayRef shape) {
    std::string s = "[";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + "]";
}

// The address of a tensor that has to be contiguous, of this shape and type, on
// device `dev`.
void* like(const char* name, const Tensor& t, IntArrayRef shape, ScalarType dt, int dev) {
    if (t.scalar_type() != dt || !t.sizes().equals(shape) || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
        throw py::value_error(std::string(name) + " must be a contiguous " + c10::toString(dt) + " " + text(shape) +
                              " tensor on cuda:" + std::to_string(dev) + ", got " + text(t));
    return t.data_ptr();
}
void* opt(const char* name, const Tensor& t, IntArrayRef shape, ScalarType dt, int dev) {
    return t.defined() ? like(name, t, shape, dt, dev) : nullptr;
}
const uint8_t* flags(const Tensor& t, IntArrayRef shape, int dev) {
    if (!t.defined()) return nullptr;
    return (const uint8_t*)like("reset", t, shape, t.scalar_type() == at::kBool ? at::kBool : at::kByte, dev);
}
// The first tensor of a call: its device.  dims < 0: any number of at least one.
int first(const char* name, const char* form, const Tensor& t, int64_t dims) {
    if (!t.is_cuda() || !t.is_contiguous() || (dims < 0 ? t.dim() < 1 : t.dim() != dims))
        throw py::value_error(std::string(name) + " must be a contiguous " + form + " CUDA tensor, got " + text(t));
    return t.get_device();
}
int code(const Tensor& t) {
    if (t.scalar_type() == at::kFloat) return LR_F32;
    if (t.scalar_type() == at::kBFloat16) return LR_BF16;
    throw py::type_error(std::string("storage dtype must be float32 or bfloat16, got ") + c10::toString(t.scalar_type()));
}
// The stream of a call: given, or the current one.  The tensors' device has to be
// the current one (the library launches there) and the stream's.
void* stream_on(const py::object& s, int dev) {
    if (dev != (int)c10::cuda::current_device())
        throw py::value_error("the tensors are on cuda:" + std::to_string(dev) + " but the current CUDA device is cuda:" +
                              std::to_string((int)c10::cuda::current_device()) + ": call under torch.cuda.device");
    if (s.is_none()) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    const int sd = s.attr("device").attr("index").cast<int>();
    if (sd != dev)
        throw py::value_error("the stream belongs to cuda:" + std::to_string(sd) + ", the tensors to cuda:" + std::to_string(dev));
    return (void*)s.attr("cuda_stream").cast<uintptr_t>();
}
// The call's stream, current while its outputs are allocated: memory that another
// stream may still be reading (the allocator's, taken back there) is none to write on it.
struct OnStream {
    void* s;
    c10::cuda::OptionalCUDAStreamGuard guard;
    OnStream(const py::object& stream, int dev) : s(stream_on(stream, dev)) {
        if (!stream.is_none())
            guard.reset_stream(c10::cuda::getStreamFromExternal((cudaStream_t)s, (c10::DeviceIndex)dev));
    }
};
void check(int st) {
    if (st == LR_OK) return;
    py::module_::import("linear_recurrence_scan_chunked_gb300").attr("_check")(st);
}
template <class F>
void call(F&& f) {
    int st;
    {
        py::gil_scoped_release nogil;
        st = f();
    }
    check(st);
}
Tensor make(const Tensor& given, IntArrayRef shape, ScalarType dt, const Tensor& ref) {
    return given.defined() ? given : at::empty(shape, ref.options().dtype(dt));
}

// ------------------------------------------------------- gated recurrence

struct GlrArgs {
    const void *x, *zr, *zi;
    const float *lam, *br, *bi;
};
GlrArgs glr_args(const Tensor& x, const Tensor& zr, const Tensor& zi, const Tensor& lam, const Tensor& br,
                 const Tensor& bi, int dev) {
    const IntArrayRef s = x.sizes(), d = s.slice(s.size() - 1);
    const ScalarType t = x.scalar_type();
    return GlrArgs{x.data_ptr(), like("zr", zr, s, t, dev), like("zi", zi, s, t, dev),
                   (const float*)like("lam", lam, d, at::kFloat, dev), (const float*)like("br", br, d, at::kFloat, dev),
                   (const float*)like("bi", bi, d, at::kFloat, dev)};
}

py::tuple p_glr_fwd(py::object x_, py::object zr, py::object zi, py::object lam, py::object br, py::object bi, py::object h0_,
                    py::object reset_, py::object h_, py::object last_, bool want_last, py::object stream) {
    const Tensor x = need("x", x_), h0 = arg("h0", h0_), reset = arg("reset", reset_);
    const int dev = first("x", "[T, B, D]", x, 3);
    const int64_t T = x.size(0), B = x.size(1), D = x.size(2);
    const IntArrayRef st = x.sizes().slice(1);
    const GlrArgs a = glr_args(x, need("zr", zr), need("zi", zi), need("lam", lam), need("br", br), need("bi", bi), dev);
    const float* p0 = (const float*)opt("h0", h0, st, at::kFloat, dev);
    const uint8_t* rs = flags(reset, x.sizes().slice(0, 2), dev);
    const int dt = code(x);
    const OnStream on(stream, dev);
    const Tensor h = make(arg("h", h_), x.sizes(), x.scalar_type(), x);
    Tensor last = arg("h_last", last_);
    if (!last.defined() && want_last) last = make(last, st, at::kFloat, x);
    void* ph = like("h", h, x.sizes(), x.scalar_type(), dev);
    float* pl = (float*)opt("h_last", last, st, at::kFloat, dev);
    call([&] { return glr_fwd(a.x, a.zr, a.zi, a.lam, a.br, a.bi, p0, rs, ph, pl, B, T, D, dt, on.s); });
    return py::make_tuple(wrap(h), wrap(last));
}

py::tuple p_glr_bwd(py::object x_, py::object zr, py::object zi, py::object lam_, py::object br, py::object bi, py::object h_,
                    py::object dh_, py::object h0_, py::object reset_, py::object dlast_, py::tuple out, bool want_dh0,
                    py::object stream) {
    const Tensor x = need("x", x_), lam = need("lam", lam_), h0 = arg("h0", h0_), reset = arg("reset", reset_),
                 dlast = arg("dh_last", dlast_);
    const int dev = first("x", "[T, B, D]", x, 3);
    const int64_t T = x.size(0), B = x.size(1), D = x.size(2);
    const IntArrayRef sq = x.sizes(), st = sq.slice(1), d = sq.slice(2);
    const ScalarType t = x.scalar_type();
    const GlrArgs a = glr_args(x, need("zr", zr), need("zi", zi), lam, need("br", br), need("bi", bi), dev);
    const float* p0 = (const float*)opt("h0", h0, st, at::kFloat, dev);
    const uint8_t* rs = flags(reset, sq.slice(0, 2), dev);
    const void* ph = like("h", need("h", h_), sq, t, dev);
    const void* pdh = like("dh", need("dh", dh_), sq, t, dev);
    const float* pdl = (const float*)opt("dh_last", dlast, st, at::kFloat, dev);
    const int dt = code(x);
    const OnStream on(stream, dev);
    static const char* names[7] = {"dx", "dzr", "dzi", "dlam", "dbr", "dbi", "dh0"};
    Tensor o[7];
    void* p[7];
    for (int k = 0; k < 7; ++k) {
        o[k] = arg(names[k], out[k]);
        const IntArrayRef shape = k < 3 ? sq : k < 6 ? d : st;
        const ScalarType type = k < 3 ? t : at::kFloat;
        if (k < 6 || want_dh0) o[k] = make(o[k], shape, type, x);
        p[k] = opt(names[k], o[k], shape, type, dev);
    }
    call([&] {
        return glr_bwd(a.x, a.zr, a.zi, a.lam, a.br, a.bi, p0, rs, ph, pdh, pdl, p[0], p[1], p[2], (float*)p[3], (float*)p[4],
                       (float*)p[5], (float*)p[6], B, T, D, dt, on.s);
    });
    return py::make_tuple(wrap(o[0]), wrap(o[1]), wrap(o[2]), wrap(o[3]), wrap(o[4]), wrap(o[5]), wrap(o[6]));
}

py::object p_glr_step(py::object x_, py::object zr, py::object zi, py::object lam, py::object br, py::object bi,
                      py::object state_, py::object slots_, py::object reset_, py::object h_, py::object stream) {
    const Tensor x = need("x", x_), state = need("state", state_), slots = arg("slots", slots_), reset = arg("reset", reset_);
    const int dev = first("x", "[B, D]", x, 2);
    const int64_t B = x.size(0), D = x.size(1);
    const GlrArgs a = glr_args(x, need("zr", zr), need("zi", zi), need("lam", lam), need("br", br), need("bi", bi), dev);
    const int64_t n_slots = state.dim() == 2 ? state.size(0) : 0;
    float* ps = (float*)like("state", state, {n_slots, D}, at::kFloat, dev);
    if (!slots.defined() && n_slots < B)
        throw py::value_error("state has " + std::to_string(n_slots) + " slots for " + std::to_string(B) + " rows");
    const uint8_t* rs = flags(reset, x.sizes().slice(0, 1), dev);
    const int32_t* psl = (const int32_t*)opt("slots", slots, x.sizes().slice(0, 1), at::kInt, dev);
    const int dt = code(x);
    const OnStream on(stream, dev);
    const Tensor h = make(arg("h", h_), x.sizes(), x.scalar_type(), x);
    void* ph = like("h", h, x.sizes(), x.scalar_type(), dev);
    call([&] { return glr_step(a.x, a.zr, a.zi, a.lam, a.br, a.bi, rs, psl, ps, ph, B, n_slots, D, dt, on.s); });
    return wrap(h);
}

// ------------------------------------------------------------- layer norm

py::tuple p_layer_norm_fwd(py::object x_, py::object w_, py::object b_, py::object res_, double eps, py::object y_,
                           py::object s_, py::object stream) {
    const Tensor x = need("x", x_), w = need("w", w_), b = arg("b", b_), res = arg("res", res_);
    const int dev = first("x", "[..., D]", x, -1);
    const IntArrayRef shape = x.sizes(), row = shape.slice(0, shape.size() - 1), d = shape.slice(shape.size() - 1);
    const ScalarType t = x.scalar_type();
    const float* pw = (const float*)like("w", w, d, at::kFloat, dev);
    const float* pb = (const float*)opt("b", b, d, at::kFloat, dev);
    const void* pr = opt("res", res, shape, t, dev);
    Tensor sum = arg("s", s_);
    if (sum.defined() && !res.defined()) throw py::value_error("s is an output of the residual add: give res with it");
    const int dt = code(x);
    const OnStream on(stream, dev);
    if (res.defined()) sum = make(sum, shape, t, x);
    const Tensor y = make(arg("y", y_), shape, t, x), mean = make(Tensor(), row, at::kFloat, x),
                 rstd = make(Tensor(), row, at::kFloat, x);
    void* py_ = like("y", y, shape, t, dev);
    void* psum = opt("s", sum, shape, t, dev);
    const int64_t N = mean.numel(), D = d[0];
    call([&] {
        return layer_norm_fwd(x.data_ptr(), pr, pw, pb, py_, psum, mean.data_ptr<float>(), rstd.data_ptr<float>(), N, D,
                              (float)eps, dt, on.s);
    });
    if (!res.defined()) return py::make_tuple(wrap(y), wrap(mean), wrap(rstd));
    return py::make_tuple(wrap(y), wrap(mean), wrap(rstd), wrap(sum));
}

py::tuple p_layer_norm_bwd(py::object x_, py::object w_, py::object mean_, py::object rstd_, py::object dy_, py::object dres_,
                           py::object dx_, py::object dw_, py::object db_, py::object stream) {
    const Tensor x = need("x", x_), w = need("w", w_), mean = need("mean", mean_), rstd = need("rstd", rstd_),
                 dres = arg("dres", dres_);
    const int dev = first("x", "[..., D]", x, -1);
    const IntArrayRef shape = x.sizes(), row = shape.slice(0, shape.size() - 1), d = shape.slice(shape.size() - 1);
    const ScalarType t = x.scalar_type();
    const float* pw = (const float*)like("w", w, d, at::kFloat, dev);
    const float* pm = (const float*)like("mean", mean, row, at::kFloat, dev);
    const float* pq = (const float*)like("rstd", rstd, row, at::kFloat, dev);
    const void* pdy = like("dy", need("dy", dy_), shape, t, dev);
    const void* pr = opt("dres", dres, shape, t, dev);
    const int dt = code(x);
    const OnStream on(stream, dev);
    const Tensor dx = make(arg("dx", dx_), shape, t, x), dw = make(arg("dw", dw_), d, at::kFloat, x),
                 db = make(arg("db", db_), d, at::kFloat, x);
    void* pdx = like("dx", dx, shape, t, dev);
    float* pdw = (float*)like("dw", dw, d, at::kFloat, dev);
    float* pdb = (float*)like("db", db, d, at::kFloat, dev);
    const int64_t N = mean.numel(), D = d[0];
    call([&] { return layer_norm_bwd(x.data_ptr(), pw, pm, pq, pdy, pr, pdx, pdw, pdb, N, D, dt, on.s); });
    return py::make_tuple(wrap(dx), wrap(dw), wrap(db));
}

// ---------------------------------------------------------- cross entropy

struct LceArgs {
    Tensor x, w, target;
    int dev;
    int64_t N, V, D;
};
LceArgs lce_args(const py::object& x_, const py::object& w_, const py::object& t_) {
    LceArgs a{need("x", x_), need("w", w_), need("target", t_), 0, 0, 0, 0};
    a.dev = first("x", "[..., D]", a.x, -1);
    a.D = a.x.size(-1);
    a.V = a.w.dim() == 2 ? a.w.size(0) : 0;
    like("w", a.w, {a.V, a.D}, a.x.scalar_type(), a.dev);
    like("target", a.target, a.x.sizes().slice(0, a.x.dim() - 1), at::kLong, a.dev);
    a.N = a.target.numel();
    return a;
}

py::tuple p_lce_fwd(py::object x_, py::object w_, py::object t_, int64_t ignore, py::object loss_, py::object lse_,
                    py::object stream) {
    const LceArgs a = lce_args(x_, w_, t_);
    const IntArrayRef row = a.target.sizes();
    const int dt = code(a.x);
    const OnStream on(stream, a.dev);
    const Tensor loss = make(arg("loss", loss_), row, at::kFloat, a.x), lse = make(arg("lse", lse_), row, at::kFloat, a.x);
    float* pl = (float*)like("loss", loss, row, at::kFloat, a.dev);
    float* pz = (float*)like("lse", lse, row, at::kFloat, a.dev);
    call([&] {
        return lce_fwd(a.x.data_ptr(), a.w.data_ptr(), a.target.data_ptr<int64_t>(), ignore, pl, pz, a.N, a.V, a.D, dt, on.s);
    });
    return py::make_tuple(wrap(loss), wrap(lse));
}

py::tuple p_lce_bwd(py::object x_, py::object w_, py::object t_, py::object lse_, py::object dloss_, int64_t ignore,
                    py::object dx_, py::object dw_, py::object stream) {
    const LceArgs a = lce_args(x_, w_, t_);
    const IntArrayRef row = a.target.sizes();
    const float* pz = (const float*)like("lse", need("lse", lse_), row, at::kFloat, a.dev);
    const float* pg = (const float*)like("dloss", need("dloss", dloss_), row, at::kFloat, a.dev);
    const ScalarType t = a.x.scalar_type();
    const int dt = code(a.x);
    const OnStream on(stream, a.dev);
    const Tensor dx = make(arg("dx", dx_), a.x.sizes(), t, a.x), dw = make(arg("dw", dw_), a.w.sizes(), t, a.x);
    void* pdx = like("dx", dx, a.x.sizes(), t, a.dev);
    void* pdw = like("dw", dw, a.w.sizes(), t, a.dev);
    call([&] {
        return lce_bwd(a.x.data_ptr(), a.w.data_ptr(), a.target.data_ptr<int64_t>(), ignore, pz, pg, pdx, pdw, a.N, a.V, a.D,
                       dt, on.s);
    });
    return py::make_tuple(wrap(dx), wrap(dw));
}

// ------------------------------------------------------------------ AdamW

// The addresses of a list of contiguous tensors of one type on device `dev`, with
// the given numbers of elements.
std::vector<void*> addresses(const char* name, const py::object& list, ScalarType dt, const std::vector<int64_t>& n, int dev,
                             bool scales = false) {
    const py::object fast = py::reinterpret_steal<py::object>(PySequence_Fast(list.ptr(), "a list of tensors is expected"));
    if (!fast) throw py::error_already_set();
    const size_t count = (size_t)PySequence_Fast_GET_SIZE(fast.ptr());
    if (count != n.size())
        throw py::value_error(std::string(name) + " has " + std::to_string(count) + " tensors, params " + std::to_string(n.size()));
    std::vector<void*> p(count);
    for (size_t i = 0; i < count; ++i) {
        PyObject* o = PySequence_Fast_GET_ITEM(fast.ptr(), (Py_ssize_t)i);
        if (!THPVariable_Check(o)) throw py::type_error(std::string(name) + " must hold tensors");
        const Tensor& t = THPVariable_Unpack(o);
        const int64_t want = scales ? (n[i] + 255) / 256 : n[i];
        if (t.scalar_type() != dt || t.numel() != want || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
            throw py::value_error(std::string(name) + "[" + std::to_string(i) + "] must be a contiguous " + c10::toString(dt) +
                                  " tensor of " + std::to_string(want) + " elements on cuda:" + std::to_string(dev) + ", got " +
                                  text(t));
        p[i] = t.data_ptr();
    }
    return p;
}
// The numbers of elements of a list's tensors, and the first one's device.
std::vector<int64_t> numels(const char* name, const py::object& list, int* dev) {
    const py::object fast = py::reinterpret_steal<py::object>(PySequence_Fast(list.ptr(), "a list of tensors is expected"));
    if (!fast) throw py::error_already_set();
    std::vector<int64_t> n((size_t)PySequence_Fast_GET_SIZE(fast.ptr()));
    for (size_t i = 0; i < n.size(); ++i) {
        PyObject* o = PySequence_Fast_GET_ITEM(fast.ptr(), (Py_ssize_t)i);
        if (!THPVariable_Check(o)) throw py::type_error(std::string(name) + " must hold tensors");
        const Tensor& t = THPVariable_Unpack(o);
        if (i == 0) {
            if (!t.is_cuda()) throw py::value_error(std::string(name) + " must hold CUDA tensors");
            *dev = t.get_device();
        }
        n[i] = t.numel();
    }
    return n;
}

void p_adamw(bool eight, py::object params, py::object grads, py::object m, py::object v, py::object ms, py::object vs,
             py::object copies, py::object grad_scale, int64_t step, double lr, double b1, double b2, double eps, double wd,
             uint32_t seed, py::object stream) {
    int dev = 0;
    const std::vector<int64_t> n = numels("params", params, &dev);
    if (n.empty()) return;
    ScalarType gt = at::kFloat;
    if (py::len(grads) > 0) {
        const py::object g0 = grads[py::int_(0)];
        gt = need("grads[0]", g0).scalar_type();
    }
    if (gt != at::kFloat && gt != at::kBFloat16)
        throw py::type_error(std::string("gradients must be float32 or bfloat16, got ") + c10::toString(gt));
    const ScalarType mt = eight ? at::kChar : at::kFloat, vt = eight ? at::kByte : at::kFloat;
    const std::vector<void*> pp = addresses("params", params, at::kFloat, n, dev), pg = addresses("grads", grads, gt, n, dev),
                             pm = addresses("m", m, mt, n, dev), pv = addresses("v", v, vt, n, dev);
    std::vector<void*> pms, pvs, pc;
    if (eight) {
        pms = addresses("ms", ms, at::kFloat, n, dev, true);
        pvs = addresses("vs", vs, at::kFloat, n, dev, true);
    }
    if (!copies.is_none()) pc = addresses("copies", copies, at::kBFloat16, n, dev);
    const Tensor gs = arg("grad_scale", grad_scale);
    const float* pgs = nullptr;
    if (gs.defined()) {
        const int64_t one[1] = {1};
        pgs = (const float*)like("grad_scale", gs, gs.numel() == 1 ? gs.sizes() : IntArrayRef(one, 1), at::kFloat, dev);
    }
    void* s = stream_on(stream, dev);
    const int gd = gt == at::kFloat ? LR_F32 : LR_BF16;
    const int64_t count = (int64_t)n.size();
    call([&] {
        void* const* c = pc.empty() ? nullptr : pc.data();
        if (eight)
            return adamw8_step(count, n.data(), (float* const*)pp.data(), (const void* const*)pg.data(),
                               (int8_t* const*)pm.data(), (uint8_t* const*)pv.data(), (float* const*)pms.data(),
                               (float* const*)pvs.data(), c, step, lr, b1, b2, eps, wd, pgs, seed, gd, s);
        return adamw_step(count, n.data(), (float* const*)pp.data(), (const void* const*)pg.data(),
                          (float* const*)pm.data(), (float* const*)pv.data(), c, step, lr, b1, b2, eps, wd, pgs, gd, s);
    });
}

void p_adamw8_values(py::object mq, py::object vq, py::object ms, py::object vs, py::object m, py::object v,
                     py::object stream) {
    int dev = 0;
    const std::vector<int64_t> n = numels("the codes", mq, &dev);
    if (n.empty()) return;
    const std::vector<void*> a = addresses("mq", mq, at::kChar, n, dev), b = addresses("vq", vq, at::kByte, n, dev),
                             c = addresses("ms", ms, at::kFloat, n, dev, true), d = addresses("vs", vs, at::kFloat, n, dev, true),
                             e = addresses("m", m, at::kFloat, n, dev), f = addresses("v", v, at::kFloat, n, dev);
    void* s = stream_on(stream, dev);
    call([&] {
        return adamw8_values((int64_t)n.size(), n.data(), (const int8_t* const*)a.data(), (const uint8_t* const*)b.data(),
                             (const float* const*)c.data(), (const float* const*)d.data(), (float* const*)e.data(),
                             (float* const*)f.data(), s);
    });
}

}  // namespace

PYBIND11_MODULE(_lrs_binding, m) {
    m.def("glr_fwd", &p_glr_fwd);
    m.def("glr_bwd", &p_glr_bwd);
    m.def("glr_step", &p_glr_step);
    m.def("layer_norm_fwd", &p_layer_norm_fwd);
    m.def("layer_norm_bwd", &p_layer_norm_bwd);
    m.def("lce_fwd", &p_lce_fwd);
    m.def("lce_bwd", &p_lce_bwd);
    m.def("adamw", &p_adamw);
    m.def("adamw8_values", &p_adamw8_values);
}
