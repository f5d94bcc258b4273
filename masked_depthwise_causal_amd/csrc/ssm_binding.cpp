// ssm_binding.cpp -- the state space block's operators on torch tensors, as a CPython module (_ssm).
//
// It checks and marshals arguments, allocates outputs and workspaces with torch, and calls the
// C-ABI of mccb_ssm.h on torch's current stream; nothing is computed here. The functions of the library
// are handed over by address (bind), so that the module works with whichever build is loaded.
// Written against torch's C++ interface because a call's cost is this marshalling: a single-token call
// takes 9-12 us with the same steps in Python, against 3 us for the launch.
#include "binding.h"
#include "mccb_ssm.h"

namespace {

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
PyObject *bind(PyObject *, PyObject *args) { return bind_to(lib, args); }

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
