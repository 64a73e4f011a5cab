// The torch-level calls of the query/key and gated feed-forward operators:
// argument checks, outputs and workspaces from torch's allocator, the current
// stream, and the library's C entry point.  Host work only, compiled because a
// small call is as long as its host part: with the same steps in Python and
// ctypes a call took 16-18 us, of which the kernels of a few tokens need 4.
//
// The entry points' addresses come from the Python package, which loads the
// library, so there is one copy of it in the process.
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include <array>
#include <optional>
#include <sstream>
#include <tuple>
#include <variant>

#include "../../include/rtlynx.h"

namespace {

namespace py = pybind11;
using at::Tensor;
using MaybeTensor = std::optional<Tensor>;
using MaybePair = std::optional<std::pair<Tensor, MaybeTensor>>;

struct {
    decltype(&rtlynx_rope) rope, rope_backward;
    decltype(&rtlynx_qk_norm_rope) norm_rope;
    decltype(&rtlynx_qk_norm_rope_backward) norm_rope_backward;
    decltype(&rtlynx_qk_norm_rope_workspace_size) norm_rope_workspace;
    decltype(&rtlynx_workspace_size) linear_workspace;
    decltype(&rtlynx_gated_mlp_block) gated;
    decltype(&rtlynx_gated_mlp_block_workspace_size) gated_workspace;
    decltype(&rtlynx_gated_mlp_backward) gated_backward;
    decltype(&rtlynx_gated_mlp_backward_workspace_size) gated_backward_workspace;
} api;

template <typename F>
void take(F& f, const py::dict& addresses, const char* name) {
    f = reinterpret_cast<F>(addresses[name].cast<uintptr_t>());
}

void bind(const py::dict& a) {
    take(api.rope, a, "rtlynx_rope");
    take(api.rope_backward, a, "rtlynx_rope_backward");
    take(api.norm_rope, a, "rtlynx_qk_norm_rope");
    take(api.norm_rope_backward, a, "rtlynx_qk_norm_rope_backward");
    take(api.norm_rope_workspace, a, "rtlynx_qk_norm_rope_workspace_size");
    take(api.linear_workspace, a, "rtlynx_workspace_size");
    take(api.gated, a, "rtlynx_gated_mlp_block");
    take(api.gated_workspace, a, "rtlynx_gated_mlp_block_workspace_size");
    take(api.gated_backward, a, "rtlynx_gated_mlp_backward");
    take(api.gated_backward_workspace, a, "rtlynx_gated_mlp_backward_workspace_size");
}

// A bad status of the library, raised in Python as RtlynxError.
struct StatusError {
    int status;
    const char* what;
};

void check(int status, const char* what) {
    if (status != RTLYNX_OK) throw StatusError{status, what};
}

template <typename... Parts>
[[noreturn]] void refuse(const Parts&... parts) {
    std::ostringstream s;
    (s << ... << parts);
    throw py::value_error(s.str());
}

std::string seen(const Tensor& t) {
    std::ostringstream s;
    s << t.scalar_type() << " " << t.sizes() << " on " << t.device();
    return s.str();
}

void* data(const MaybeTensor& t) { return t ? t->data_ptr() : nullptr; }

Tensor bytes(size_t n, const Tensor& like) {
    return at::empty({static_cast<int64_t>(n)}, like.options().dtype(at::kByte));
}

// ---------------------------------------------------------------- query and key heads
// [S, H, D] or [B, S, H, D], any strides but contiguous channels.
struct Heads {
    int64_t B, S, D;
    int dtype;

    explicit Heads(const Tensor& q) {
        const int64_t n = q.dim();
        if (!q.is_cuda() || (n != 3 && n != 4)) refuse("CUDA tensors [S, H, D] or [B, S, H, D], got ", seen(q));
        B = n == 4 ? q.size(0) : 1;
        S = q.size(n - 3);
        D = q.size(n - 1);
        switch (q.scalar_type()) {
            case at::kBFloat16: dtype = RTLYNX_BF16; break;
            case at::kHalf: dtype = RTLYNX_FP16; break;
            case at::kFloat: dtype = RTLYNX_FP32; break;
            default: refuse("bf16, fp16 or fp32 tensors, got ", seen(q));
        }
    }
};

// View of t, which has q's shape but for the heads (those of `like` if given).
rtlynx_heads view(const Tensor& t, const Tensor& q, const Tensor* like, const char* what) {
    const int64_t n = q.dim();
    bool ok = t.scalar_type() == q.scalar_type() && t.device() == q.device() && t.dim() == n;
    for (int64_t i = 0; ok && i < n; ++i)
        if (i != n - 2) ok = t.size(i) == q.size(i);
    if (ok && like) ok = t.size(n - 2) == like->size(n - 2);
    if (!ok) refuse(what, ": ", seen(t), " does not go with ", seen(like ? *like : q));
    if (t.stride(n - 1) != 1 && t.size(n - 1) > 1)
        refuse(what, ": the channels of a head are contiguous, got strides ", t.strides());
    return {t.data_ptr(), t.size(n - 2), n == 4 ? t.stride(0) : 0, t.stride(n - 3), t.stride(n - 2)};
}

struct Positions {
    const rtlynx_rope_spec* spec;
    const void* data;
    int64_t b, s, a;
};

// positions [S, axes], shared by the sequences, or [B, S, axes]; `specs` is the
// address of three specs, one for each rtlynx_pos_type.
Positions positions_of(const Tensor& p, uintptr_t specs, int64_t axes, const Tensor& q, const Heads& h) {
    Positions r{reinterpret_cast<const rtlynx_rope_spec*>(specs), p.data_ptr(), 0, 0, 0};
    int kind = -1;
    if (p.scalar_type() == at::kInt) kind = RTLYNX_POS_INT32;
    if (p.scalar_type() == at::kLong) kind = RTLYNX_POS_INT64;
    if (p.scalar_type() == at::kFloat) kind = RTLYNX_POS_FP32;
    if (kind < 0 || p.device() != q.device()) refuse("positions: int32, int64 or float32 on ", q.device(), ", got ", seen(p));
    r.spec += kind;
    const int64_t n = p.dim();
    const bool own = n == 3 && p.size(0) == h.B;
    if ((n != 2 && !own) || p.size(n - 2) != h.S || p.size(n - 1) != axes)
        refuse("positions: [", h.S, ", ", axes, "] or [", h.B, ", ", h.S, ", ", axes, "], got ", seen(p));
    if (own) r.b = p.stride(0);
    r.s = p.stride(n - 2);
    r.a = p.stride(n - 1);
    return r;
}

const void* weight(const MaybeTensor& w, const Tensor& q, const char* what) {
    if (!w) return nullptr;
    if (w->dim() != 1 || w->size(0) != q.size(-1) || w->scalar_type() != q.scalar_type() || w->device() != q.device() ||
        !w->is_contiguous())
        refuse(what, ": contiguous [", q.size(-1), "] of ", q.dtype(), " on ", q.device(), ", got ", seen(*w));
    return w->data_ptr();
}

// Queries, and keys where there are any, with their views.
struct Pair {
    Tensor q;
    MaybeTensor k;
    rtlynx_heads qv, kv;
    const rtlynx_heads* keys() const { return k ? &kv : nullptr; }
};

Pair inputs(const Tensor& q, const MaybeTensor& k, const Tensor& first, const Tensor* like_q, const Tensor* like_k,
            const char* q_name, const char* k_name) {
    Pair p{q, k, view(q, first, like_q, q_name), {}};
    if (k) p.kv = view(*k, first, like_k, k_name);
    return p;
}

// `out`, or new contiguous tensors of the shapes of q and k.
Pair outputs(const MaybePair& out, const Tensor& q, const MaybeTensor& k) {
    if (out) {
        if (k.has_value() != out->second.has_value()) refuse("out: queries and keys as in the call");
        return inputs(out->first, out->second, q, &q, k ? &*k : nullptr, "q_out", "k_out");
    }
    const auto plain = at::MemoryFormat::Contiguous;
    Tensor qo = at::empty_like(q, q.options(), plain);
    MaybeTensor ko;
    if (k) ko = at::empty_like(*k, k->options(), plain);
    return inputs(qo, ko, q, nullptr, nullptr, "q_out", "k_out");
}

std::tuple<Tensor, MaybeTensor> rope(bool backward, const Tensor& q, const MaybeTensor& k, const Tensor& positions, uintptr_t specs, int64_t axes,
               const MaybePair& out) {
    const Heads h(q);
    const c10::cuda::CUDAGuard guard(q.device());
    const Pair in = inputs(q, k, q, nullptr, nullptr, "q", "k");
    const Positions p = positions_of(positions, specs, axes, q, h);
    const Pair o = outputs(out, q, k);
    check((backward ? api.rope_backward : api.rope)(&in.qv, in.keys(), &o.qv, o.keys(), h.B, h.S, h.D, h.dtype, p.spec,
                                                    p.data, p.b, p.s, p.a,
                                                    c10::cuda::getCurrentCUDAStream(q.get_device()).stream()),
          backward ? "rtlynx_rope_backward" : "rtlynx_rope");
    return {o.q, o.k};
}

std::tuple<Tensor, MaybeTensor> qk_norm_rope(const Tensor& q, const MaybeTensor& k, const MaybeTensor& w_q, const MaybeTensor& w_k,
                       const Tensor& positions, uintptr_t specs, int64_t axes, double eps, const MaybePair& out) {
    const Heads h(q);
    const c10::cuda::CUDAGuard guard(q.device());
    const Pair in = inputs(q, k, q, nullptr, nullptr, "q", "k");
    const Positions p = positions_of(positions, specs, axes, q, h);
    const void *wq = weight(w_q, q, "w_q"), *wk = weight(w_k, q, "w_k");
    const Pair o = outputs(out, q, k);
    check(api.norm_rope(&in.qv, in.keys(), wq, wk, &o.qv, o.keys(), h.B, h.S, h.D, h.dtype, static_cast<float>(eps), p.spec,
                        p.data, p.b, p.s, p.a, c10::cuda::getCurrentCUDAStream(q.get_device()).stream()),
          "rtlynx_qk_norm_rope");
    return {o.q, o.k};
}

using HeadGrads = std::tuple<Tensor, MaybeTensor, MaybeTensor, MaybeTensor>;
HeadGrads qk_norm_rope_backward(const Tensor& dq_out, const MaybeTensor& dk_out, const Tensor& q, const MaybeTensor& k,
                                const MaybeTensor& w_q, const MaybeTensor& w_k, const Tensor& positions, uintptr_t specs,
                                int64_t axes, double eps, const MaybePair& out, bool weight_grads) {
    const Heads h(q);
    const c10::cuda::CUDAGuard guard(q.device());
    if (k.has_value() != dk_out.has_value()) refuse("dk_out goes with k");
    const Pair in = inputs(q, k, q, nullptr, nullptr, "q", "k");
    const Pair grads = inputs(dq_out, dk_out, q, &q, k ? &*k : nullptr, "dq_out", "dk_out");
    const Positions p = positions_of(positions, specs, axes, q, h);
    const void *wq = weight(w_q, q, "w_q"), *wk = weight(w_k, q, "w_k");
    const Pair o = outputs(out, q, k);
    MaybeTensor dw_q, dw_k, ws;
    if (weight_grads && w_q) dw_q = at::empty({h.D}, q.options().dtype(at::kFloat));
    if (weight_grads && w_k && k) dw_k = at::empty({h.D}, q.options().dtype(at::kFloat));
    size_t n = 0;
    if (dw_q || dw_k) {
        n = api.norm_rope_workspace(h.D);
        ws = bytes(n, q);
    }
    check(api.norm_rope_backward(&grads.qv, grads.keys(), &in.qv, in.keys(), wq, wk, &o.qv, o.keys(),
                                 static_cast<float*>(data(dw_q)), static_cast<float*>(data(dw_k)), h.B, h.S, h.D, h.dtype,
                                 static_cast<float>(eps), p.spec, p.data, p.b, p.s, p.a, data(ws), n,
                                 c10::cuda::getCurrentCUDAStream(q.get_device()).stream()),
          "rtlynx_qk_norm_rope_backward");
    return {o.q, o.k, dw_q, dw_k};
}

// ---------------------------------------------------------------- gated feed-forward block
// The address of a contiguous [rows, cols] matrix of this type on X's device.
void* matrix(const Tensor& t, int64_t rows, int64_t cols, const Tensor& X, const char* what,
             at::ScalarType type = at::kBFloat16) {
    if (t.scalar_type() != type || t.device() != X.device() || t.dim() != 2 || t.size(0) != rows || t.size(1) != cols ||
        !t.is_contiguous())
        refuse(what, ": contiguous ", type, " [", rows, ", ", cols, "] on ", X.device(), ", got ", seen(t));
    return t.data_ptr();
}

struct Gated {
    int64_t M, D, F;
    void *x, *gate, *up, *down;

    Gated(const Tensor& X, const Tensor& W_gate, const Tensor& W_up, const Tensor& W_down) {
        if (!X.is_cuda() || X.dim() != 2 || W_gate.dim() != 2) refuse("X [M, D] and W_gate [D_ff, D] are CUDA matrices");
        M = X.size(0), D = X.size(1), F = W_gate.size(0);
        x = matrix(X, M, D, X, "X");
        gate = matrix(W_gate, F, D, X, "W_gate");
        up = matrix(W_up, F, D, X, "W_up");
        down = matrix(W_down, D, F, X, "W_down");
    }
};

// mode: none given is the dense down-projection, where a LoRA pair would be
// left out without a word; asked for by name, the dense one leaves it out as
// the linear layer's does.
using Saved = std::tuple<Tensor, Tensor, Tensor, Tensor>;
std::variant<Tensor, std::tuple<Tensor, Saved>> gated_mlp(const Tensor& X, const Tensor& W_gate, const Tensor& W_up, const Tensor& W_down, int act,
                     const MaybeTensor& L_A, const MaybeTensor& L_B, const std::optional<int>& mode, bool save,
                     const MaybeTensor& out) {
    if (!mode && (L_A || L_B)) refuse("L_A and L_B belong to mode_down=MODE_SPARSE, no mode_down given");
    const int mode_down = mode.value_or(RTLYNX_MODE_DENSE_SKIP);
    const bool lora = mode_down != RTLYNX_MODE_DENSE_SKIP && (L_A || L_B);
    if (lora && !(L_A && L_B)) refuse("one of L_A and L_B without the other");
    if (lora && L_B->dim() != 2) refuse("L_B: a matrix [R, D_ff], got ", seen(*L_B));
    const Gated g(X, W_gate, W_up, W_down);
    const c10::cuda::CUDAGuard guard(X.device());
    const int64_t R = lora ? L_B->size(0) : 0;
    const void* la = lora ? matrix(*L_A, g.D, R, X, "L_A") : nullptr;
    const void* lb = lora ? matrix(*L_B, R, g.F, X, "L_B") : nullptr;
    const Tensor Y = out ? *out : at::empty_like(X);
    void* y = matrix(Y, g.M, g.D, X, "out");
    const Tensor H = at::empty({g.M, g.F}, X.options());
    MaybeTensor G, U, low, ws;
    if (save) {
        G = at::empty({g.M, g.F}, X.options());
        U = at::empty({g.M, g.F}, X.options());
        low = at::empty({g.M, g.F}, X.options().dtype(at::kShort));
    }
    const size_t n = mode_down == RTLYNX_MODE_SPARSE ? api.linear_workspace(g.M, g.F, g.D, R, mode_down)
                                                     : api.gated_workspace(g.M, g.D, g.F, mode_down);
    if (n) ws = bytes(n, X);
    check(api.gated(g.x, g.gate, g.up, g.down, la, lb, data(G), data(U), data(low), H.data_ptr(), y, g.M, g.D, g.F, R, act,
                    mode_down, data(ws), n, c10::cuda::getCurrentCUDAStream(X.get_device()).stream()),
          "rtlynx_gated_mlp_block");
    if (!save) return Y;
    return std::tuple<Tensor, Saved>(Y, Saved(*G, *U, *low, H));
}

using GatedGrads = std::tuple<MaybeTensor, MaybeTensor, MaybeTensor, MaybeTensor>;
GatedGrads gated_mlp_backward(const Tensor& dY, const Tensor& X, const Tensor& W_gate, const Tensor& W_up,
                              const Tensor& W_down, const Saved& saved, int act, const std::array<bool, 4>& needs) {
    const Gated g(X, W_gate, W_up, W_down);
    const c10::cuda::CUDAGuard guard(X.device());
    const void* dy = matrix(dY, g.M, g.D, X, "dY");
    const void* G = matrix(std::get<0>(saved), g.M, g.F, X, "G");
    const void* U = matrix(std::get<1>(saved), g.M, g.F, X, "U");
    const void* low = matrix(std::get<2>(saved), g.M, g.F, X, "low", at::kShort);
    const void* H = matrix(std::get<3>(saved), g.M, g.F, X, "H");
    const Tensor* of[4] = {&X, &W_gate, &W_up, &W_down};
    MaybeTensor d[4];
    for (int i = 0; i < 4; ++i)
        if (needs[i]) d[i] = at::empty_like(*of[i]);
    const size_t n = api.gated_backward_workspace(g.M, g.D, g.F);
    const Tensor ws = bytes(n, X);
    check(api.gated_backward(dy, g.x, g.gate, g.up, g.down, G, U, low, H, data(d[0]), data(d[1]), data(d[2]), data(d[3]), g.M,
                             g.D, g.F, act, ws.data_ptr(), n, c10::cuda::getCurrentCUDAStream(X.get_device()).stream()),
          "rtlynx_gated_mlp_backward");
    return {d[0], d[1], d[2], d[3]};
}

}  // namespace

PYBIND11_MODULE(rtlynx_torch, m) {
    py::register_exception_translator([](std::exception_ptr p) {
        try {
            if (p) std::rethrow_exception(p);
        } catch (const StatusError& e) {
            const py::object cls = py::module_::import("activation_sparse_gemm_b200").attr("RtlynxError");
            PyErr_SetObject(cls.ptr(), cls(e.status, e.what).ptr());
        }
    });
    m.def("bind", &bind);
    // Without Python's lock from the arguments' conversion to the results': a
    // launch waits where the stream's queue is full, and torch's allocator may.
    using Unlocked = py::call_guard<py::gil_scoped_release>;
    m.def("rope", &rope, Unlocked());
    m.def("qk_norm_rope", &qk_norm_rope, Unlocked());
    m.def("qk_norm_rope_backward", &qk_norm_rope_backward, Unlocked());
    m.def("gated_mlp", &gated_mlp, Unlocked());
    m.def("gated_mlp_backward", &gated_mlp_backward, Unlocked());
}
