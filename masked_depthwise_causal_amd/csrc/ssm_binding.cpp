// ssm_binding.cpp -- the state space block's operators on torch tensors, as a CPython module (_ssm).
//
// It checks and marshals arguments, allocates outputs and workspaces with torch, and calls the
// C-ABI of mccb_ssm.h on torch's current stream; nothing is computed here. The functions of the library
// are handed over by address (bind), so that the module works with whichever build is loaded.
// Written against torch's C++ interface because a call's cost is this marshalling: a single-token call
// takes 9-12 us with the same steps in Python, against 3 us for the launch.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <cstring>
#include <string>

#include "mccb_ssm.h"

namespace {

using at::Tensor;
using Shape = at::IntArrayRef;

// The library's functions, in the order in which bind takes their addresses.
struct Library {
    decltype(&mccb_conv_act_forward) conv_forward;
    decltype(&mccb_conv_act_backward_get_workspace_size) conv_backward_size;
    decltype(&mccb_conv_act_backward) conv_backward;
    decltype(&mccb_conv_act_step) conv_step;
    decltype(&mccb_scan_saved_size) scan_saved_size;
    decltype(&mccb_scan_forward_get_workspace_size) scan_forward_size;
    decltype(&mccb_scan_forward) scan_forward;
    decltype(&mccb_scan_backward_get_workspace_size) scan_backward_size;
    decltype(&mccb_scan_backward) scan_backward;
    decltype(&mccb_scan_step) scan_step;
    decltype(&mccb_linear_forward_get_workspace_size) linear_forward_size;
    decltype(&mccb_linear_forward) linear_forward;
    decltype(&mccb_linear_backward_get_workspace_size) linear_backward_size;
    decltype(&mccb_linear_backward) linear_backward;
};
Library lib{};
constexpr Py_ssize_t kFunctions = sizeof(Library) / sizeof(void *);
PyObject *error_class = nullptr;  // MccbError(status, where)

// A status that is not MCCB_OK, on its way to Python.
struct Status {
    int code;
    const char *where;
};
void ok(int code, const char *where) {
    if (code != MCCB_OK) throw Status{code, where};
}

// -- arguments ------------------------------------------------------------------------------------
Tensor tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) TORCH_CHECK_TYPE(false, name, " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}
Tensor maybe(PyObject *o, const char *name) { return o == Py_None ? Tensor() : tensor(o, name); }

std::string text(Shape s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

void check(const char *name, const Tensor &t, Shape shape, at::ScalarType type, at::Device device,
           bool contiguous) {
    TORCH_CHECK_VALUE(t.device() == device, name, " must live on ", device.str(), " (a HIP device)");
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " has shape ", text(t.sizes()), ", expected ", text(shape));
    TORCH_CHECK_VALUE(t.scalar_type() == type, name, " has dtype ", toString(t.scalar_type()),
                      ", expected ", toString(type));
    if (contiguous) TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
}
void check_if(const char *name, const Tensor &t, Shape shape, at::ScalarType type, at::Device device,
              bool contiguous = true) {
    if (t.defined()) check(name, t, shape, type, device, contiguous);
}

// The tensor that sets a call's type and device.
int32_t kind_of(const char *name, const Tensor &t, int64_t dims, const char *layout) {
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must live on a HIP device");
    TORCH_CHECK_VALUE(t.dim() == dims, name, " must be ", layout);
    if (t.scalar_type() == at::kBFloat16) return MCCB_BF16;
    TORCH_CHECK_VALUE(t.scalar_type() == at::kHalf, "dtype ", toString(t.scalar_type()),
                      " not supported (bfloat16, float16)");
    return MCCB_FP16;
}

void *ptr(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }
void strides3(const Tensor &t, int64_t (&s)[3], bool token) {
    if (!t.defined()) return;
    const auto v = t.strides();
    if (token) s[0] = 0, s[1] = v[0], s[2] = v[1];
    else s[0] = v[0], s[1] = v[1], s[2] = v[2];
}
// Strides along S, B, G, N of B or C, whose group axis may be left out.
void strides4(const Tensor &t, int64_t (&s)[4], bool token, bool grouped) {
    const auto v = t.strides();
    size_t i = 0;
    s[0] = token ? 0 : v[i++];
    s[1] = v[i++];
    s[2] = grouped ? v[i++] : 0;
    s[3] = v[i];
}

void *stream_of(const Tensor &t) { return (void *)c10::hip::getCurrentHIPStream(t.device().index()).stream(); }

Tensor make(Shape shape, const Tensor &like) { return at::empty(shape, like.options()); }
Tensor make(Shape shape, const Tensor &like, at::ScalarType type) {
    return at::empty(shape, like.options().dtype(type));
}
Tensor bytes(uint64_t n, const Tensor &like) {
    return n ? make({(int64_t)n}, like, at::kByte) : Tensor();
}

// Tensors of the caller's that a call wrote: their version moves on, as an in-place operation's does.
void wrote(std::initializer_list<Tensor> ts) {
    for (const Tensor &t : ts)
        if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

PyObject *out(const Tensor &t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
PyObject *tuple(std::initializer_list<Tensor> ts) {
    PyObject *r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) return nullptr;
    Py_ssize_t i = 0;
    for (const Tensor &t : ts) PyTuple_SET_ITEM(r, i++, out(t));
    return r;
}

// -- convolution ----------------------------------------------------------------------------------
struct Conv {
    mccb_conv_t a{};
    Tensor x, weight, bias, lengths, state;
    c10::hip::OptionalHIPGuard here;  // launches go to the current device: make it x's
};

void conv_args(Conv &c, PyObject *x, PyObject *weight, PyObject *bias, long act, bool token) {
    c.x = tensor(x, "x");
    c.a.dtype = kind_of("x", c.x, token ? 2 : 3, token ? "[B,H]" : "[S,B,H]");
    c.here.set_index(c.x.device().index());
    c.weight = tensor(weight, "weight");
    TORCH_CHECK_VALUE(c.weight.dim() == 2, "weight must be a [W,H] tensor");
    c.bias = maybe(bias, "bias");
    const auto s = c.x.sizes();
    c.a.S = token ? 1 : s[0];
    c.a.B = s[s.size() - 2], c.a.H = s[s.size() - 1], c.a.W = c.weight.size(0);
    c.a.activation = (int32_t)act;
    const auto type = c.x.scalar_type();
    const auto device = c.x.device();
    check("weight", c.weight, {c.a.W, c.a.H}, type, device, true);
    check_if("bias", c.bias, {c.a.H}, type, device);
    c.a.x = ptr(c.x);
    strides3(c.x, c.a.x_stride, token);
    c.a.weight = ptr(c.weight), c.a.bias = ptr(c.bias);
}
void conv_rows(Conv &c, PyObject *lengths, PyObject *state) {
    c.lengths = maybe(lengths, "lengths"), c.state = maybe(state, "state");
    check_if("lengths", c.lengths, {c.a.B}, at::kLong, c.x.device());
    check_if("state", c.state, {c.a.W - 1, c.a.B, c.a.H}, c.x.scalar_type(), c.x.device());
    c.a.lengths = (const int64_t *)ptr(c.lengths), c.a.state = ptr(c.state);
}

// (x, weight, bias, act, lengths, state, return_state, y, final_state)
PyObject *conv_forward(PyObject *const *v) {
    Conv c;
    conv_args(c, v[0], v[1], v[2], PyLong_AsLong(v[3]), false);
    conv_rows(c, v[4], v[5]);
    const bool with_state = v[6] == Py_True;
    Tensor y = maybe(v[7], "y"), final_state = maybe(v[8], "final_state");
    const auto type = c.x.scalar_type();
    if (y.defined()) check("y", y, c.x.sizes(), type, c.x.device(), true);
    else y = make(c.x.sizes(), c.x);
    const std::array<int64_t, 3> carried{c.a.W - 1, c.a.B, c.a.H};
    check_if("final_state", final_state, carried, type, c.x.device());
    if (with_state && !final_state.defined()) final_state = make(carried, c.x);
    ok(lib.conv_forward(&c.a, ptr(y), ptr(final_state), stream_of(c.x)), "mccb_conv_act_forward");
    wrote({y, final_state});
    return with_state ? tuple({y, final_state}) : out(y);
}

// (gradY, x, weight, bias, act, lengths, state, gradFinalState)
PyObject *conv_backward(PyObject *const *v) {
    Conv c;
    conv_args(c, v[1], v[2], v[3], PyLong_AsLong(v[4]), false);
    conv_rows(c, v[5], v[6]);
    const Tensor gy = tensor(v[0], "gradY"), gfinal = maybe(v[7], "gradFinalState");
    const auto type = c.x.scalar_type();
    const std::array<int64_t, 3> carried{c.a.W - 1, c.a.B, c.a.H};
    check("gradY", gy, c.x.sizes(), type, c.x.device(), false);
    check_if("gradFinalState", gfinal, carried, type, c.x.device());
    uint64_t n = 0;
    ok(lib.conv_backward_size(&c.a, &n), "mccb_conv_act_backward_get_workspace_size");
    const Tensor gx = make(c.x.sizes(), c.x), gw = make(c.weight.sizes(), c.x);
    const Tensor gb = c.bias.defined() ? make(c.bias.sizes(), c.x) : Tensor();
    const Tensor gs = c.state.defined() ? make(carried, c.x) : Tensor();
    const Tensor ws = bytes(n, c.x);
    int64_t gy_stride[3];
    strides3(gy, gy_stride, false);
    ok(lib.conv_backward(&c.a, ptr(gy), gy_stride, ptr(gfinal), ptr(gx), ptr(gw), ptr(gb), ptr(gs),
                         ptr(ws), n, stream_of(c.x)),
       "mccb_conv_act_backward");
    return tuple({gx, gw, gb, gs});
}

// (x, weight, state, bias, act, y)
PyObject *conv_step(PyObject *const *v) {
    Conv c;
    conv_args(c, v[0], v[1], v[3], PyLong_AsLong(v[4]), true);
    const Tensor state = tensor(v[2], "state");
    const auto type = c.x.scalar_type();
    check("state", state, {c.a.W - 1, c.a.B, c.a.H}, type, c.x.device(), true);
    Tensor y = maybe(v[5], "y");
    if (y.defined()) check("y", y, c.x.sizes(), type, c.x.device(), true);
    else y = make(c.x.sizes(), c.x);
    ok(lib.conv_step(&c.a, ptr(state), ptr(y), stream_of(c.x)), "mccb_conv_act_step");
    wrote({state, y});
    return out(y);
}

// -- scan -----------------------------------------------------------------------------------------
struct Scan {
    mccb_scan_t a{};
    Tensor x, dt, A, B, C, D, z, bias, lengths, state;
    c10::hip::OptionalHIPGuard here;
};

// v: x, dt, A, B, C, D, z, dt_bias, softplus
void scan_args(Scan &c, PyObject *const *v, bool token) {
    c.x = tensor(v[0], "x");
    c.a.dtype = kind_of("x", c.x, token ? 2 : 3, token ? "[B,H]" : "[S,B,H]");
    c.here.set_index(c.x.device().index());
    c.dt = tensor(v[1], "dt"), c.A = tensor(v[2], "A"), c.B = tensor(v[3], "B"), c.C = tensor(v[4], "C");
    c.D = maybe(v[5], "D"), c.z = maybe(v[6], "z"), c.bias = maybe(v[7], "dt_bias");
    const auto rows = c.x.sizes();
    const auto type = c.x.scalar_type();
    const auto device = c.x.device();
    const int64_t dims = (int64_t)rows.size();
    mccb_scan_t &a = c.a;
    a.S = token ? 1 : rows[0];
    a.B = rows[dims - 2], a.H = rows[dims - 1];
    TORCH_CHECK_VALUE(c.A.dim() == 2, "A must be a [N,H] tensor");
    a.N = c.A.size(0);
    const bool grouped = c.B.dim() == dims + 1;
    TORCH_CHECK_VALUE(grouped || c.B.dim() == dims,
                      "B and C must be [S,B,N] or [S,B,G,N] ([B,N] or [B,G,N] for one token)");
    a.G = grouped ? c.B.size(dims - 1) : 1;
    at::DimVector coef(rows.begin(), rows.end() - 1);
    if (grouped) coef.push_back(a.G);
    coef.push_back(a.N);
    check("dt", c.dt, rows, type, device, false);
    check_if("z", c.z, rows, type, device, false);
    check("A", c.A, {a.N, a.H}, at::kFloat, device, true);
    check("B", c.B, coef, type, device, false);
    check("C", c.C, coef, type, device, false);
    check_if("D", c.D, {a.H}, at::kFloat, device);
    check_if("dt_bias", c.bias, {a.H}, at::kFloat, device);
    a.softplus = v[8] == Py_True;
    a.x = ptr(c.x), a.dt = ptr(c.dt), a.z = ptr(c.z), a.Bm = ptr(c.B), a.Cm = ptr(c.C);
    strides3(c.x, a.x_stride, token);
    strides3(c.dt, a.dt_stride, token);
    strides3(c.z, a.z_stride, token);
    strides4(c.B, a.b_stride, token, grouped);
    strides4(c.C, a.c_stride, token, grouped);
    a.A = (const float *)ptr(c.A), a.D = (const float *)ptr(c.D), a.dt_bias = (const float *)ptr(c.bias);
}
void scan_rows(Scan &c, PyObject *lengths, PyObject *state) {
    c.lengths = maybe(lengths, "lengths"), c.state = maybe(state, "state");
    check_if("lengths", c.lengths, {c.a.B}, at::kLong, c.x.device());
    check_if("state", c.state, {c.a.B, c.a.N, c.a.H}, at::kFloat, c.x.device());
    c.a.lengths = (const int64_t *)ptr(c.lengths), c.a.state = (const float *)ptr(c.state);
}
int64_t saved_floats(const Scan &c) {
    uint64_t n = 0;
    ok(lib.scan_saved_size(&c.a, &n), "mccb_scan_saved_size");
    return (int64_t)(n / sizeof(float));
}

// (x, dt, A, B, C, D, z, dt_bias, softplus, lengths, state, return_state, return_saved, out, final_state)
PyObject *scan_forward(PyObject *const *v) {
    Scan c;
    scan_args(c, v, false);
    scan_rows(c, v[9], v[10]);
    const bool with_state = v[11] == Py_True, with_saved = v[12] == Py_True;
    Tensor y = maybe(v[13], "out"), final_state = maybe(v[14], "final_state"), saved;
    if (y.defined()) check("out", y, c.x.sizes(), c.x.scalar_type(), c.x.device(), true);
    else y = make(c.x.sizes(), c.x);
    const std::array<int64_t, 3> states{c.a.B, c.a.N, c.a.H};
    check_if("final_state", final_state, states, at::kFloat, c.x.device());
    if (with_state && !final_state.defined()) final_state = make(states, c.x, at::kFloat);
    if (with_saved) saved = make({saved_floats(c)}, c.x, at::kFloat);
    uint64_t n = 0;
    ok(lib.scan_forward_size(&c.a, &n), "mccb_scan_forward_get_workspace_size");
    const Tensor ws = bytes(n, c.x);
    ok(lib.scan_forward(&c.a, ptr(y), (float *)ptr(final_state), ptr(saved), ptr(ws), n, stream_of(c.x)),
       "mccb_scan_forward");
    wrote({y, final_state});
    if (with_state) return with_saved ? tuple({y, final_state, saved}) : tuple({y, final_state});
    return with_saved ? tuple({y, saved}) : out(y);
}

// (x, dt, A, B, C, D, z, dt_bias, softplus, lengths, state, gradOut, saved, gradFinalState)
PyObject *scan_backward(PyObject *const *v) {
    Scan c;
    scan_args(c, v, false);
    scan_rows(c, v[9], v[10]);
    const Tensor go = tensor(v[11], "gradOut"), saved = tensor(v[12], "saved");
    const Tensor gfinal = maybe(v[13], "gradFinalState");
    const auto rows = c.x.sizes();
    const std::array<int64_t, 3> states{c.a.B, c.a.N, c.a.H};
    check("gradOut", go, rows, c.x.scalar_type(), c.x.device(), false);
    check("saved", saved, {saved_floats(c)}, at::kFloat, c.x.device(), true);
    check_if("gradFinalState", gfinal, states, at::kFloat, c.x.device());
    uint64_t n = 0;
    ok(lib.scan_backward_size(&c.a, &n), "mccb_scan_backward_get_workspace_size");
    const Tensor gx = make(rows, c.x), gdt = make(rows, c.x), gA = make(c.A.sizes(), c.A);
    const Tensor gB = make(c.B.sizes(), c.x), gC = make(c.C.sizes(), c.x);
    const Tensor gD = c.D.defined() ? make(c.D.sizes(), c.D) : Tensor();
    const Tensor gz = c.z.defined() ? make(rows, c.x) : Tensor();
    const Tensor gbias = c.bias.defined() ? make(c.bias.sizes(), c.bias) : Tensor();
    const Tensor gstate = c.state.defined() ? make(states, c.state) : Tensor();
    const Tensor ws = bytes(n, c.x);
    mccb_scan_grads_t g{};
    g.gradOut = ptr(go);
    strides3(go, g.gout_stride, false);
    g.gradFinalState = (const float *)ptr(gfinal);
    g.gradX = ptr(gx), g.gradDt = ptr(gdt), g.gradZ = ptr(gz), g.gradB = ptr(gB), g.gradC = ptr(gC);
    g.gradA = (float *)ptr(gA), g.gradD = (float *)ptr(gD), g.gradDtBias = (float *)ptr(gbias);
    g.gradState = (float *)ptr(gstate);
    ok(lib.scan_backward(&c.a, &g, ptr(saved), ptr(ws), n, stream_of(c.x)), "mccb_scan_backward");
    return tuple({gx, gdt, gA, gB, gC, gD, gz, gbias, gstate});
}

// (x, dt, A, B, C, D, z, dt_bias, softplus, state, out)
PyObject *scan_step(PyObject *const *v) {
    Scan c;
    scan_args(c, v, true);
    const Tensor state = tensor(v[9], "state");
    check("state", state, {c.a.B, c.a.N, c.a.H}, at::kFloat, c.x.device(), true);
    Tensor y = maybe(v[10], "out");
    if (y.defined()) check("out", y, c.x.sizes(), c.x.scalar_type(), c.x.device(), true);
    else y = make(c.x.sizes(), c.x);
    ok(lib.scan_step(&c.a, (float *)ptr(state), ptr(y), stream_of(c.x)), "mccb_scan_step");
    wrote({state, y});
    return out(y);
}

// -- matrix product -------------------------------------------------------------------------------
// A [...,C] tensor as R evenly spaced, contiguous rows.
void rows_of(const char *name, const Tensor &t, int64_t &R, int64_t &ld) {
    const auto size = t.sizes(), stride = t.strides();
    const int64_t last = t.dim() - 1, C = size[last];
    TORCH_CHECK_VALUE(C <= 1 || stride[last] == 1, name, "'s last dimension must be contiguous");
    R = 1, ld = -1;
    for (int64_t i = last - 1; i >= 0; --i) {
        if (size[i] != 1) {
            if (ld < 0) ld = stride[i];
            else TORCH_CHECK_VALUE(size[i] == 0 || R == 0 || stride[i] == ld * R, name,
                                   "'s rows are not evenly spaced: make it contiguous");
        }
        R *= size[i];
    }
    if (ld < 0) ld = C;
}

struct Linear {
    mccb_linear_t a{};
    Tensor x, weight, bias;
    at::DimVector shape;  // of the output
    c10::hip::OptionalHIPGuard here;
};

void linear_args(Linear &c, PyObject *x, PyObject *weight, PyObject *bias, long act) {
    c.x = tensor(x, "x");
    TORCH_CHECK_VALUE(c.x.dim() >= 2, "x must be a [...,K] tensor of at least two dimensions");
    rows_of("x", c.x, c.a.M, c.a.x_ld);
    c.a.dtype = kind_of("x", c.x, c.x.dim(), "[...,K]");
    c.here.set_index(c.x.device().index());
    c.a.K = c.x.size(-1);
    c.weight = tensor(weight, "weight");
    TORCH_CHECK_VALUE(c.weight.dim() == 2, "weight must be a [N,K] tensor");
    c.a.N = c.weight.size(0);
    check("weight", c.weight, {c.a.N, c.a.K}, c.x.scalar_type(), c.x.device(), false);
    int64_t n;
    rows_of("weight", c.weight, n, c.a.weight_ld);
    c.bias = maybe(bias, "bias");
    check_if("bias", c.bias, {c.a.N}, c.x.scalar_type(), c.x.device());
    c.a.activation = (int32_t)act;
    c.a.x = ptr(c.x), c.a.weight = ptr(c.weight), c.a.bias = ptr(c.bias);
    c.shape.assign(c.x.sizes().begin(), c.x.sizes().end());
    c.shape.back() = c.a.N;
}

// (x, weight, bias, act, residual, return_pre, out, whether pre is fp32)
PyObject *linear_forward(PyObject *const *v) {
    Linear c;
    linear_args(c, v[0], v[1], v[2], PyLong_AsLong(v[3]));
    const auto type = c.x.scalar_type();
    const Tensor residual = maybe(v[4], "residual");
    int64_t rows, residual_ld = 0;
    if (residual.defined()) {
        check("residual", residual, c.shape, type, c.x.device(), false);
        rows_of("residual", residual, rows, residual_ld);
    }
    Tensor y = maybe(v[6], "out"), pre;
    if (y.defined()) check("out", y, c.shape, type, c.x.device(), true);
    else y = make(c.shape, c.x);
    c.a.pre_fp32 = v[7] == Py_True;
    if (v[5] == Py_True) pre = make(c.shape, c.x, c.a.pre_fp32 ? at::kFloat : type);
    uint64_t n = 0;
    ok(lib.linear_forward_size(&c.a, &n), "mccb_linear_forward_get_workspace_size");
    const Tensor ws = bytes(n, c.x);
    ok(lib.linear_forward(&c.a, ptr(residual), residual_ld, ptr(y), ptr(pre), ptr(ws), n, stream_of(c.x)),
       "mccb_linear_forward");
    wrote({y});
    return pre.defined() ? tuple({y, pre}) : out(y);
}

// (gradOut, x, weight, pre, act, grad_x, grad_weight, grad_bias)
PyObject *linear_backward(PyObject *const *v) {
    Linear c;
    linear_args(c, v[1], v[2], Py_None, PyLong_AsLong(v[4]));
    const auto type = c.x.scalar_type();
    const Tensor go = tensor(v[0], "gradOut"), pre = maybe(v[3], "pre");
    check("gradOut", go, c.shape, type, c.x.device(), false);
    int64_t rows, go_ld;
    rows_of("gradOut", go, rows, go_ld);
    c.a.pre_fp32 = pre.defined() && pre.scalar_type() == at::kFloat;
    check_if("pre", pre, c.shape, c.a.pre_fp32 ? at::kFloat : type, c.x.device());
    uint64_t n = 0;
    ok(lib.linear_backward_size(&c.a, &n), "mccb_linear_backward_get_workspace_size");
    const Tensor gx = v[5] == Py_True ? make(c.x.sizes(), c.x) : Tensor();
    const Tensor gw = v[6] == Py_True ? make({c.a.N, c.a.K}, c.x) : Tensor();
    const Tensor gb = v[7] == Py_True ? make({c.a.N}, c.x) : Tensor();
    const Tensor ws = bytes(n, c.x);
    ok(lib.linear_backward(&c.a, ptr(go), go_ld, ptr(pre), ptr(gx), ptr(gw), ptr(gb), ptr(ws), n,
                           stream_of(c.x)),
       "mccb_linear_backward");
    return tuple({gx, gw, gb});
}

// -- the module -----------------------------------------------------------------------------------
// Every entry checks the argument count and turns what is thrown into a Python exception.
template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *entry(PyObject *, PyObject *const *v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N || !error_class) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", n, N);
        return nullptr;
    }
    try {
        PyObject *r = F(v);
        if (PyErr_Occurred()) {
            Py_XDECREF(r);
            return nullptr;
        }
        return r;
    } catch (const Status &s) {
        PyObject *e = PyObject_CallFunction(error_class, "is", s.code, s.where);
        if (e) {
            PyErr_SetObject(error_class, e);
            Py_DECREF(e);
        }
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// bind(error class, addresses)
PyObject *bind(PyObject *, PyObject *args) {
    PyObject *cls, *addresses;
    if (!PyArg_ParseTuple(args, "OO!", &cls, &PyTuple_Type, &addresses)) return nullptr;
    if (PyTuple_GET_SIZE(addresses) != kFunctions) {
        PyErr_SetString(PyExc_ValueError, "wrong number of functions");
        return nullptr;
    }
    void *table[kFunctions];
    for (Py_ssize_t i = 0; i < kFunctions; ++i) {
        table[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(addresses, i));
        if (!table[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a function has no address");
            return nullptr;
        }
    }
    static_assert(sizeof(table) == sizeof(lib), "a table of function pointers");
    std::memcpy(&lib, table, sizeof(lib));
    Py_INCREF(cls);
    Py_XSETREF(error_class, cls);
    Py_RETURN_NONE;
}

#define ENTRY(name, n) {#name, (PyCFunction)(void *)&entry<name, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"bind", &bind, METH_VARARGS, nullptr},
    ENTRY(conv_forward, 9),
    ENTRY(conv_backward, 8),
    ENTRY(conv_step, 6),
    ENTRY(scan_forward, 15),
    ENTRY(scan_backward, 14),
    ENTRY(scan_step, 11),
    ENTRY(linear_forward, 8),
    ENTRY(linear_backward, 8),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ssm", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ssm() { return PyModule_Create(&module); }
