// delta_binding.cpp -- the gated delta rule and the norms around a block on torch tensors, as a CPython module
// (_delta): checks and marshals arguments, allocates outputs and workspaces with torch, and calls the C-ABI
// of mccb_delta.h on torch's current stream; nothing is computed here. The functions of the library are
// handed over by address (bind), so that the module works with whichever build is loaded.
#include <cmath>

#include "binding.h"
#include "mccb_delta.h"

namespace {

// The library's functions, in the order in which bind takes their addresses.
struct Library {
    decltype(&mccb_delta_saved_size) delta_saved_size;
    decltype(&mccb_delta_forward_get_workspace_size) delta_forward_size;
    decltype(&mccb_delta_forward) delta_forward;
    decltype(&mccb_delta_backward_get_workspace_size) delta_backward_size;
    decltype(&mccb_delta_backward) delta_backward;
    decltype(&mccb_delta_step) delta_step;
    decltype(&mccb_prenorm_forward) prenorm_forward;
    decltype(&mccb_prenorm_backward_get_workspace_size) prenorm_backward_size;
    decltype(&mccb_prenorm_backward) prenorm_backward;
    decltype(&mccb_postnorm_forward) postnorm_forward;
    decltype(&mccb_postnorm_backward_get_workspace_size) postnorm_backward_size;
    decltype(&mccb_postnorm_backward) postnorm_backward;
};
Library lib{};

// -- gated delta rule -----------------------------------------------------------------------------
struct Delta {
    mccb_delta_t a{};
    Tensor q, k, v, dt, b, A, bias, lengths, state;
    c10::hip::OptionalHIPGuard here;  // launches go to the current device: make it q's
};

// A tensor [S,B,heads,width] ([B,heads,width] for one token) whose rows are contiguous, and its strides.
void head_rows(const char *name, const Tensor &t, Shape shape, const Tensor &like, int64_t (&s)[3], bool token) {
    check(name, t, shape, like.scalar_type(), like.device(), false);
    TORCH_CHECK_VALUE(t.size(-1) <= 1 || t.stride(-1) == 1, name, "'s last dimension must be contiguous");
    strides3(t, s, token);
}

// v: q, k, v, dt, b, A, dt_bias, softplus, normalize, scale
void delta_args(Delta &c, PyObject *const *v, bool token) {
    c.q = tensor(v[0], "q");
    c.a.dtype = kind_of("q", c.q, token ? 3 : 4, token ? "[B,G,K]" : "[S,B,G,K]");
    c.here.set_index(c.q.device().index());
    c.k = tensor(v[1], "k"), c.v = tensor(v[2], "v"), c.dt = tensor(v[3], "dt"), c.b = tensor(v[4], "b");
    c.A = tensor(v[5], "A"), c.bias = maybe(v[6], "dt_bias");
    const auto size = c.q.sizes();
    const size_t lead = token ? 0 : 1;
    mccb_delta_t &a = c.a;
    a.S = token ? 1 : size[0];
    a.B = size[lead], a.G = size[lead + 1], a.K = size[lead + 2];
    TORCH_CHECK_VALUE(c.v.dim() == c.q.dim(), "v must be ", token ? "[B,H,V]" : "[S,B,H,V]");
    a.H = c.v.size(-2), a.V = c.v.size(-1);
    at::DimVector rows(size.begin(), size.begin() + lead + 1), values = rows;
    rows.push_back(a.H);
    values.push_back(a.H), values.push_back(a.V);
    head_rows("q", c.q, size, c.q, a.q_stride, token);
    head_rows("k", c.k, size, c.q, a.k_stride, token);
    head_rows("v", c.v, values, c.q, a.v_stride, token);
    const auto type = c.q.scalar_type();
    const auto device = c.q.device();
    check("dt", c.dt, rows, type, device, false);
    check("b", c.b, rows, type, device, false);
    strides3(c.dt, a.dt_stride, token);
    strides3(c.b, a.b_stride, token);
    check("A", c.A, {a.H}, at::kFloat, device, true);
    check_if("dt_bias", c.bias, {a.H}, at::kFloat, device);
    a.softplus = v[7] == Py_True, a.normalize = v[8] == Py_True;
    a.scale = v[9] == Py_None ? (float)(1.0 / std::sqrt((double)(a.K > 0 ? a.K : 1))) : (float)PyFloat_AsDouble(v[9]);
    a.q = ptr(c.q), a.k = ptr(c.k), a.v = ptr(c.v), a.dt = ptr(c.dt), a.b = ptr(c.b);
    a.A = (const float *)ptr(c.A), a.dt_bias = (const float *)ptr(c.bias);
}
void delta_rows(Delta &c, PyObject *lengths, PyObject *state) {
    c.lengths = maybe(lengths, "lengths"), c.state = maybe(state, "state");
    check_if("lengths", c.lengths, {c.a.B}, at::kLong, c.q.device());
    check_if("state", c.state, {c.a.B, c.a.H, c.a.K, c.a.V}, at::kFloat, c.q.device());
    c.a.lengths = (const int64_t *)ptr(c.lengths), c.a.state = (const float *)ptr(c.state);
}
int64_t saved_bytes(const Delta &c) {
    uint64_t n = 0;
    ok(lib.delta_saved_size(&c.a, &n), "mccb_delta_saved_size");
    return (int64_t)n;
}

// (q, k, v, dt, b, A, dt_bias, softplus, normalize, scale, lengths, state, return_state, return_saved, out, final_state)
PyObject *delta_forward(PyObject *const *v) {
    Delta c;
    delta_args(c, v, false);
    delta_rows(c, v[10], v[11]);
    const bool with_state = v[12] == Py_True, with_saved = v[13] == Py_True;
    Tensor y = maybe(v[14], "out"), final_state = maybe(v[15], "final_state"), saved;
    if (y.defined()) check("out", y, c.v.sizes(), c.v.scalar_type(), c.v.device(), true);
    else y = make(c.v.sizes(), c.v);
    const std::array<int64_t, 4> states{c.a.B, c.a.H, c.a.K, c.a.V};
    check_if("final_state", final_state, states, at::kFloat, c.v.device());
    if (with_state && !final_state.defined()) final_state = make(states, c.v, at::kFloat);
    uint64_t n = 0;
    if (with_saved) saved = make({saved_bytes(c)}, c.v, at::kByte);
    else ok(lib.delta_forward_size(&c.a, &n), "mccb_delta_forward_get_workspace_size");
    const Tensor ws = bytes(n, c.v);
    ok(lib.delta_forward(&c.a, ptr(y), (float *)ptr(final_state), ptr(saved), ptr(ws), n, stream_of(c.v)),
       "mccb_delta_forward");
    wrote({y, final_state});
    if (with_state) return with_saved ? tuple({y, final_state, saved}) : tuple({y, final_state});
    return with_saved ? tuple({y, saved}) : out(y);
}

// (q, k, v, dt, b, A, dt_bias, softplus, normalize, scale, lengths, state, gradOut, saved, gradFinalState)
PyObject *delta_backward(PyObject *const *v) {
    Delta c;
    delta_args(c, v, false);
    delta_rows(c, v[10], v[11]);
    const Tensor go = tensor(v[12], "gradOut"), saved = tensor(v[13], "saved");
    const Tensor gfinal = maybe(v[14], "gradFinalState");
    const std::array<int64_t, 4> states{c.a.B, c.a.H, c.a.K, c.a.V};
    mccb_delta_grads_t g{};
    head_rows("gradOut", go, c.v.sizes(), c.q, g.gout_stride, false);
    check("saved", saved, {saved_bytes(c)}, at::kByte, c.q.device(), true);
    check_if("gradFinalState", gfinal, states, at::kFloat, c.q.device());
    uint64_t n = 0;
    ok(lib.delta_backward_size(&c.a, &n), "mccb_delta_backward_get_workspace_size");
    const Tensor gq = make(c.q.sizes(), c.q), gk = make(c.k.sizes(), c.q), gv = make(c.v.sizes(), c.q);
    const Tensor gdt = make(c.dt.sizes(), c.q), gb = make(c.b.sizes(), c.q), gA = make(c.A.sizes(), c.A);
    const Tensor gbias = c.bias.defined() ? make(c.bias.sizes(), c.bias) : Tensor();
    const Tensor gstate = c.state.defined() ? make(states, c.state) : Tensor();
    const Tensor ws = bytes(n, c.q);
    g.gradOut = ptr(go), g.gradFinalState = (const float *)ptr(gfinal);
    g.gradQ = ptr(gq), g.gradK = ptr(gk), g.gradV = ptr(gv), g.gradDt = ptr(gdt), g.gradB = ptr(gb);
    g.gradA = (float *)ptr(gA), g.gradDtBias = (float *)ptr(gbias), g.gradState = (float *)ptr(gstate);
    ok(lib.delta_backward(&c.a, &g, ptr(saved), ptr(ws), n, stream_of(c.q)), "mccb_delta_backward");
    return tuple({gq, gk, gv, gdt, gb, gA, gbias, gstate});
}

// (q, k, v, dt, b, A, dt_bias, softplus, normalize, scale, state, out)
PyObject *delta_step(PyObject *const *v) {
    Delta c;
    delta_args(c, v, true);
    const Tensor state = tensor(v[10], "state");
    check("state", state, {c.a.B, c.a.H, c.a.K, c.a.V}, at::kFloat, c.q.device(), true);
    Tensor y = maybe(v[11], "out");
    if (y.defined()) check("out", y, c.v.sizes(), c.v.scalar_type(), c.v.device(), true);
    else y = make(c.v.sizes(), c.v);
    ok(lib.delta_step(&c.a, (float *)ptr(state), ptr(y), stream_of(c.v)), "mccb_delta_step");
    wrote({state, y});
    return out(y);
}

// -- norms ----------------------------------------------------------------------------------------
struct Norm {
    mccb_norm_t a{};
    Tensor x, weight, residual, scale, z;
    c10::hip::OptionalHIPGuard here;
};

void norm_args(Norm &c, PyObject *x, PyObject *weight, PyObject *residual, PyObject *scale, PyObject *z,
               int64_t groups, double eps) {
    c.x = tensor(x, "x");
    TORCH_CHECK_VALUE(c.x.dim() >= 2, "x must be a [...,H] tensor of at least two dimensions");
    c.a.dtype = kind_of("x", c.x, c.x.dim(), "[...,H]");
    c.here.set_index(c.x.device().index());
    rows_of("x", c.x, c.a.R, c.a.x_ld);
    const auto type = c.x.scalar_type();
    const auto device = c.x.device();
    c.a.H = c.x.size(-1), c.a.groups = groups, c.a.eps = (float)eps;
    TORCH_CHECK_VALUE(groups >= 1 && c.a.H % groups == 0, "groups must divide H");
    c.weight = tensor(weight, "weight");
    c.a.weight_shared = groups > 1 && c.weight.dim() == 1 && c.weight.size(0) == c.a.H / groups;
    check("weight", c.weight, {c.a.weight_shared ? c.a.H / groups : c.a.H}, type, device, true);
    c.residual = maybe(residual, "residual"), c.scale = maybe(scale, "scale"), c.z = maybe(z, "z");
    check_if("scale", c.scale, {c.a.H}, type, device);
    int64_t rows;
    check_if("residual", c.residual, c.x.sizes(), type, device, false);
    if (c.residual.defined()) rows_of("residual", c.residual, rows, c.a.residual_ld);
    check_if("z", c.z, c.x.sizes(), type, device, false);
    if (c.z.defined()) rows_of("z", c.z, rows, c.a.z_ld);
    c.a.x = ptr(c.x), c.a.weight = ptr(c.weight), c.a.residual = ptr(c.residual);
    c.a.scale = ptr(c.scale), c.a.z = ptr(c.z);
}
// A result [...,H], the caller's or a new one.
Tensor norm_out(const char *name, PyObject *o, const Norm &c) {
    Tensor t = maybe(o, name);
    if (t.defined()) check(name, t, c.x.sizes(), c.x.scalar_type(), c.x.device(), true);
    else t = make(c.x.sizes(), c.x);
    return t;
}
int64_t gradient_rows(const char *name, const Tensor &t, const Norm &c) {
    int64_t rows, ld;
    check(name, t, c.x.sizes(), c.x.scalar_type(), c.x.device(), false);
    rows_of(name, t, rows, ld);
    return ld;
}

// (x, weight, residual, scale, eps, return_sum, out, sum_out)
PyObject *prenorm_forward(PyObject *const *v) {
    Norm c;
    norm_args(c, v[0], v[1], v[2], v[3], Py_None, 1, PyFloat_AsDouble(v[4]));
    const bool with_sum = v[5] == Py_True;
    const Tensor y = norm_out("out", v[6], c);
    Tensor sum;
    if (v[7] != Py_None || (with_sum && (c.residual.defined() || c.scale.defined()))) sum = norm_out("sum_out", v[7], c);
    ok(lib.prenorm_forward(&c.a, ptr(y), ptr(sum), stream_of(c.x)), "mccb_prenorm_forward");
    wrote({y, sum});
    return with_sum ? tuple({y, sum.defined() ? sum : c.x}) : out(y);
}

// (gradOut, x, weight, residual, scale, eps, gradSum)
PyObject *prenorm_backward(PyObject *const *v) {
    Norm c;
    norm_args(c, v[1], v[2], v[3], v[4], Py_None, 1, PyFloat_AsDouble(v[5]));
    const Tensor go = tensor(v[0], "gradOut"), gsum = maybe(v[6], "gradSum");
    const int64_t go_ld = gradient_rows("gradOut", go, c);
    const int64_t gsum_ld = gsum.defined() ? gradient_rows("gradSum", gsum, c) : 0;
    uint64_t n = 0;
    ok(lib.prenorm_backward_size(&c.a, &n), "mccb_prenorm_backward_get_workspace_size");
    const Tensor gx = make(c.x.sizes(), c.x), gw = make(c.weight.sizes(), c.x), ws = bytes(n, c.x);
    const Tensor gs = c.scale.defined() ? make(c.scale.sizes(), c.x) : Tensor();
    const Tensor gr = c.residual.defined() && c.scale.defined() ? make(c.x.sizes(), c.x) : Tensor();
    ok(lib.prenorm_backward(&c.a, ptr(go), go_ld, ptr(gsum), gsum_ld, ptr(gx), ptr(gr), ptr(gw), ptr(gs), ptr(ws), n,
                            stream_of(c.x)),
       "mccb_prenorm_backward");
    return tuple({gx, gw, c.residual.defined() && !gr.defined() ? gx : gr, gs});
}

// (x, weight, z, residual, scale, groups, eps, out)
PyObject *postnorm_forward(PyObject *const *v) {
    Norm c;
    norm_args(c, v[0], v[1], v[3], v[4], v[2], PyLong_AsLongLong(v[5]), PyFloat_AsDouble(v[6]));
    const Tensor y = norm_out("out", v[7], c);
    ok(lib.postnorm_forward(&c.a, ptr(y), stream_of(c.x)), "mccb_postnorm_forward");
    wrote({y});
    return out(y);
}

// (gradOut, x, weight, z, scale, groups, eps)
PyObject *postnorm_backward(PyObject *const *v) {
    Norm c;
    norm_args(c, v[1], v[2], Py_None, v[4], v[3], PyLong_AsLongLong(v[5]), PyFloat_AsDouble(v[6]));
    const Tensor go = tensor(v[0], "gradOut");
    const int64_t go_ld = gradient_rows("gradOut", go, c);
    uint64_t n = 0;
    ok(lib.postnorm_backward_size(&c.a, &n), "mccb_postnorm_backward_get_workspace_size");
    const Tensor gx = make(c.x.sizes(), c.x), gw = make(c.weight.sizes(), c.x), ws = bytes(n, c.x);
    const Tensor gz = c.z.defined() ? make(c.x.sizes(), c.x) : Tensor();
    const Tensor gs = c.scale.defined() ? make(c.scale.sizes(), c.x) : Tensor();
    ok(lib.postnorm_backward(&c.a, ptr(go), go_ld, ptr(gx), ptr(gz), ptr(gw), ptr(gs), ptr(ws), n, stream_of(c.x)),
       "mccb_postnorm_backward");
    return tuple({gx, gw, gz, gs});
}

// -- the module -----------------------------------------------------------------------------------
PyObject *bind(PyObject *, PyObject *args) { return bind_to(lib, args); }

PyMethodDef methods[] = {
    {"bind", &bind, METH_VARARGS, nullptr},
    ENTRY(delta_forward, 16),
    ENTRY(delta_backward, 15),
    ENTRY(delta_step, 12),
    ENTRY(prenorm_forward, 8),
    ENTRY(prenorm_backward, 7),
    ENTRY(postnorm_forward, 8),
    ENTRY(postnorm_backward, 7),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_delta", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__delta() { return PyModule_Create(&module); }
