// The operators around the ternary linear layers as torch autograd functions
// over the C ABI (include/bitnet.h): layer norm, 8-bit activation checkpoints,
// the gated activation, the TTQ layer with its input kept in 8 bits, and the
// linear layer with cross entropy.
//
// Only checks of arguments, allocation of outputs and workspaces, and calls of
// libbitnet.so on the tensors' device and its current stream. They are C++
// because the layers' calls are short: a step's forward and backward of a layer
// norm of 4096 x 2560 is 40 us on the GPU, and the same functions written in
// Python took 130 us of host time a step (the autograd engine runs a GPU
// node's backward on its own thread, where Python code runs cold).

#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/hip/HIPGraphsC10Utils.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/jit/frontend/tracer.h>
#include <torch/extension.h>

#include <unordered_set>
#include <vector>

#include "bitnet.h"

namespace {

using at::Tensor;
using std::optional;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;

void check(bitnet_status st) { TORCH_CHECK(st == BITNET_OK, "libbitnet: ", bitnet_status_string(st)); }

// The device made current and its current stream.
struct On {
  c10::DeviceGuard guard;
  void* stream;
  explicit On(const Tensor& t)
      : guard(t.device()), stream(c10::hip::getCurrentHIPStream(t.device().index()).stream()) {}
};

bool is_value(at::ScalarType t) { return t == at::kBFloat16 || t == at::kFloat; }
bitnet_dtype code(at::ScalarType t) { return t == at::kFloat ? BITNET_F32 : BITNET_BF16; }

void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
uint16_t* bf16(const Tensor& t) { return static_cast<uint16_t*>(ptr(t)); }
float* f32(const Tensor& t) { return static_cast<float*>(ptr(t)); }
int8_t* i8(const Tensor& t) { return static_cast<int8_t*>(ptr(t)); }

Tensor scratch(size_t bytes, const Tensor& like) {
  return at::empty({static_cast<int64_t>(bytes)}, like.options().dtype(at::kByte));
}

// t [..., K] as contiguous rows [M][K].
Tensor rows(const Tensor& t) {
  return (t.dim() == 2 ? t : t.reshape({-1, t.size(-1)})).contiguous();
}

// t contiguous, starting at a multiple of 16 bytes.
Tensor aligned(const Tensor& t) {
  Tensor c = t.contiguous();
  return reinterpret_cast<uintptr_t>(c.data_ptr()) % 16 == 0 ? c : c.clone();
}

// What every backward refuses: a second derivative, and being captured into a
// graph while a gradient goes on to a node of the default stream, at once or
// through other nodes (a view, a module's parametrization), which no capture
// can take in. Such a node is the accumulator of a leaf of which a graph made
// on the default stream is still alive, or one made there before the capture.
void check_backward() {
  TORCH_CHECK(!at::GradMode::is_enabled(), "this operator's gradients cannot be differentiated again");
  if (c10::hip::currentStreamCaptureStatusMayInitCtx() == c10::hip::CaptureStatus::None) return;
  std::vector<const torch::autograd::Node*> todo{torch::autograd::get_current_node().get()};
  std::unordered_set<const torch::autograd::Node*> seen(todo.begin(), todo.end());
  while (!todo.empty()) {
    const torch::autograd::Node* node = todo.back();
    todo.pop_back();
    for (size_t i = 0; i < node->num_outputs(); ++i) {
      const torch::autograd::Edge& e = node->next_edge(i);
      if (!e.is_valid() || !node->task_should_compute_output(i)) continue;
      const optional<c10::Stream> s = e.function->stream();
      TORCH_CHECK(!s.has_value() || s->id() != c10::hip::getDefaultHIPStream(s->device_index()).id(),
                  "a backward pass is being captured whose gradient goes to a node of the default stream: free the "
                  "results of earlier calls that use the same leaves (or make them on another stream) first");
      if (seen.insert(e.function.get()).second) todo.push_back(e.function.get());
    }
  }
}

bool is_tracing() {
  using c10::impl::TorchDispatchModeKey;
  using c10::impl::TorchDispatchModeTLS;
  if (torch::jit::tracer::isTracing()) return true;
  if (!TorchDispatchModeTLS::any_modes_set()) return false;
  for (const auto k : {TorchDispatchModeKey::FAKE, TorchDispatchModeKey::PROXY, TorchDispatchModeKey::FUNCTIONAL})
    if (TorchDispatchModeTLS::get_mode(k).has_value()) return true;
  return false;
}

// What every function refuses: being traced (the kernels' launches are in no
// trace, which would hold the allocation of the outputs alone), a tangent of
// forward-mode differentiation (which would be dropped) and tensors without
// memory, such as fake, functional and wrapped ones: what data_ptr() gives of
// a fake one is its offset in bytes, which a kernel would read as an address.
void check_eager(const char* what, std::initializer_list<const Tensor*> ts) {
  TORCH_CHECK_NOT_IMPLEMENTED(!is_tracing(), what, ": cannot be traced");
  const bool forward = c10::AutogradState::get_tls_state().get_fw_grad_mode();
  for (const Tensor* t : ts) {
    if (!t->defined()) continue;
    TORCH_CHECK_NOT_IMPLEMENTED(!forward || !t->_fw_grad(0).defined(), what, ": no forward-mode derivative");
    TORCH_CHECK_NOT_IMPLEMENTED(t->has_storage() && (t->numel() == 0 || t->storage().data() != nullptr), what,
                                ": a tensor without memory");
  }
}

bool wants_grad(std::initializer_list<const Tensor*> ts) {
  if (!at::GradMode::is_enabled()) return false;
  for (const Tensor* t : ts)
    if (t->defined() && t->requires_grad()) return true;
  return false;
}

void check_activation(const char* what, const Tensor& x) {
  TORCH_CHECK_VALUE(x.dim() >= 1 && x.size(-1) >= 1, what, " needs a last dimension of at least 1, got ", x.sizes());
  TORCH_CHECK_VALUE(x.is_cuda(), what, ": must be a GPU tensor");
}

// --- 8-bit checkpoints ---------------------------------------------------------

std::pair<Tensor, Tensor> empty_codes(int64_t M, int64_t K, const Tensor& like) {
  const int64_t Kc = bitnet_ckpt_pad(K);
  return {at::empty({M, Kc}, like.options().dtype(at::kChar)), at::empty({M, Kc / 128}, like.options().dtype(at::kFloat))};
}

std::pair<Tensor, Tensor> compress(const Tensor& x) {
  check_eager("compress", {&x});
  TORCH_CHECK_TYPE(is_value(x.scalar_type()), "compress expects bf16 or float32, got ", x.scalar_type());
  check_activation("compress", x);
  at::NoGradGuard off;
  const Tensor x2 = rows(x);
  const int64_t M = x2.size(0), K = x2.size(1);
  auto c = empty_codes(M, K, x2);
  if (M > 0) {
    On on(x2);
    check(bitnet_ckpt_pack(ptr(x2), code(x2.scalar_type()), M, K, i8(c.first), f32(c.second), on.stream));
  }
  return c;
}

Tensor decompress(const Tensor& codes, const Tensor& scales, int64_t K, at::ScalarType dtype) {
  check_eager("decompress", {&codes, &scales});
  TORCH_CHECK_TYPE(is_value(dtype), "decompress gives bf16 or float32, not ", dtype);
  TORCH_CHECK_TYPE(codes.scalar_type() == at::kChar && scales.scalar_type() == at::kFloat,
                   "codes: expected int8 and scales float32, got ", codes.scalar_type(), " and ", scales.scalar_type());
  TORCH_CHECK_VALUE(K >= 1 && codes.dim() == 2 && codes.size(1) == bitnet_ckpt_pad(K) && scales.dim() == 2 &&
                        scales.size(0) == codes.size(0) && scales.size(1) == codes.size(1) / 128,
                    "codes and scales: not a checkpoint of rows of ", K, ": ", codes.sizes(), " and ", scales.sizes());
  TORCH_CHECK_VALUE(codes.is_cuda() && scales.device() == codes.device(), "codes and scales: must be GPU tensors of one device");
  const int64_t M = codes.size(0);
  const Tensor q = codes.contiguous(), s = scales.contiguous();
  Tensor x = at::empty({M, K}, codes.options().dtype(dtype));
  if (M > 0) {
    On on(q);
    check(bitnet_ckpt_unpack(i8(q), f32(s), M, K, ptr(x), code(dtype), on.stream));
  }
  return x;
}

// --- layer norm ------------------------------------------------------------------

struct Norm {
  Tensor x2, w, b;
  int64_t M, K;
  bitnet_dtype pd = BITNET_F32;
  Norm(const Tensor& x, const Tensor& weight, const Tensor& bias) : x2(rows(x)), M(x2.size(0)), K(x2.size(1)) {
    if (weight.defined()) w = weight.contiguous();
    if (bias.defined()) b = bias.contiguous();
    if (w.defined()) pd = code(w.scalar_type());
    else if (b.defined()) pd = code(b.scalar_type());
  }
  void forward(const Tensor& y, double eps, float* mean, float* rstd, int8_t* codes, float* scales) const {
    if (M == 0) return;
    On on(x2);
    check(bitnet_layernorm_fwd(ptr(x2), code(x2.scalar_type()), ptr(w), ptr(b), pd, M, K, static_cast<float>(eps), ptr(y),
                               code(y.scalar_type()), mean, rstd, codes, scales, on.stream));
  }
};

struct LayerNormFn : torch::autograd::Function<LayerNormFn> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const optional<Tensor>& weight,
                        const optional<Tensor>& bias, double eps, at::ScalarType out, bool checkpoint) {
    const Norm n(x, weight.value_or(Tensor()), bias.value_or(Tensor()));
    Tensor y = at::empty(x.sizes(), x.options().dtype(out));
    Tensor stats = at::empty({2, n.M}, x.options().dtype(at::kFloat));  // mu, r
    Tensor codes, scales;
    if (checkpoint) std::tie(codes, scales) = empty_codes(n.M, n.K, n.x2);
    n.forward(y, eps, f32(stats), f32(stats) + n.M, i8(codes), f32(scales));
    ctx->save_for_backward({checkpoint ? Tensor() : n.x2, codes, scales, n.w, stats});
    ctx->saved_data["shape"] = x.sizes();
    ctx->saved_data["x"] = static_cast<int64_t>(x.scalar_type());
    ctx->saved_data["y"] = static_cast<int64_t>(out);
    ctx->saved_data["p"] = static_cast<int64_t>(n.pd);
    ctx->saved_data["w"] = weight.has_value();
    ctx->saved_data["b"] = bias.has_value();
    return y;
  }

  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    check_backward();
    const variable_list saved = ctx->get_saved_variables();
    const Tensor &x2 = saved[0], &codes = saved[1], &scales = saved[2], &w = saved[3], &stats = saved[4];
    const std::vector<int64_t> shape = ctx->saved_data["shape"].toIntVector();
    const auto xt = static_cast<at::ScalarType>(ctx->saved_data["x"].toInt());
    const auto yt = static_cast<at::ScalarType>(ctx->saved_data["y"].toInt());
    const auto pd = static_cast<bitnet_dtype>(ctx->saved_data["p"].toInt());
    const bool has_w = ctx->saved_data["w"].toBool(), has_b = ctx->saved_data["b"].toBool();
    const bool need_x = ctx->needs_input_grad(0);
    const bool need_w = has_w && ctx->needs_input_grad(1), need_b = has_b && ctx->needs_input_grad(1 + has_w);
    const Tensor dY = rows(grads[0].to(yt));
    const int64_t M = dY.size(0), K = dY.size(1);
    const auto po = dY.options().dtype(pd == BITNET_F32 ? at::kFloat : at::kBFloat16);
    Tensor dX, dw, db, ws;
    if (need_x) dX = at::empty(shape, dY.options().dtype(xt));
    if (M == 0) {
      if (need_w) dw = at::zeros({K}, po);
      if (need_b) db = at::zeros({K}, po);
    } else {
      size_t bytes = 0;
      if (need_w) dw = at::empty({K}, po);
      if (need_b) db = at::empty({K}, po);
      if (need_w || need_b) {
        bytes = bitnet_layernorm_workspace_bytes(M, K);
        ws = scratch(bytes, dY);
      }
      On on(dY);
      check(bitnet_layernorm_bwd(ptr(dY), code(yt), ptr(x2), code(xt), i8(codes), f32(scales), ptr(w), pd, f32(stats),
                                 f32(stats) + M, M, K, ptr(dX), ptr(dw), ptr(db), ptr(ws), bytes, on.stream));
    }
    return {dX, dw, db, Tensor(), Tensor(), Tensor()};
  }
};

Tensor layer_norm(const Tensor& x, const optional<Tensor>& weight, const optional<Tensor>& bias, double eps,
                  at::ScalarType out, bool checkpoint) {
  const Tensor w = weight.value_or(Tensor()), b = bias.value_or(Tensor());
  check_eager("layer_norm", {&x, &w, &b});
  TORCH_CHECK_TYPE(is_value(x.scalar_type()), "layer_norm expects bf16 or float32 activations, got ", x.scalar_type());
  TORCH_CHECK_TYPE(is_value(out), "out_dtype: expected bfloat16 or float32, got ", out);
  check_activation("layer_norm", x);
  for (const Tensor* p : {&w, &b}) {
    if (!p->defined()) continue;
    TORCH_CHECK_TYPE(is_value(p->scalar_type()), "weight and bias: expected bf16 or float32, got ", p->scalar_type());
    TORCH_CHECK_VALUE(p->dim() == 1 && p->size(0) == x.size(-1), "weight and bias: expected shape [", x.size(-1),
                      "], got ", p->sizes());
    TORCH_CHECK_VALUE(p->device() == x.device(), "weight and bias: on ", p->device(), ", expected ", x.device());
  }
  TORCH_CHECK_TYPE(!w.defined() || !b.defined() || w.scalar_type() == b.scalar_type(),
                   "weight and bias: one dtype expected, got ", w.defined() ? w.scalar_type() : out, " and ",
                   b.defined() ? b.scalar_type() : out);
  if (wants_grad({&x, &w, &b})) return LayerNormFn::apply(x, weight, bias, eps, out, checkpoint);
  const Norm n(x, w, b);
  Tensor y = at::empty(x.sizes(), x.options().dtype(out));
  n.forward(y, eps, nullptr, nullptr, nullptr, nullptr);
  return y;
}

// --- gated activation --------------------------------------------------------------

// t [..., K] as rows at one stride, in place where they are (the halves of a
// [..., 2K] tensor).
Tensor strided_rows(const Tensor& t) {
  Tensor r = t.dim() == 2 ? t : t.reshape({-1, t.size(-1)});
  if ((r.size(1) > 1 && r.stride(1) != 1) || (r.size(0) > 1 && r.stride(0) < r.size(1))) r = r.contiguous();
  return r;
}
int64_t row_stride(const Tensor& r) { return r.defined() && r.size(0) > 1 ? r.stride(0) : r.defined() ? r.size(1) : 0; }

// The checkpoints of gate and up in one buffer.
struct GateCodes {
  int8_t *gq = nullptr, *uq = nullptr;
  float *gs = nullptr, *us = nullptr;
  static size_t half(int64_t M, int64_t K) {
    const size_t n = static_cast<size_t>(M) * bitnet_ckpt_pad(K);
    return (n + n / 32 + 255) / 256 * 256;
  }
  GateCodes() = default;
  GateCodes(const Tensor& buffer, int64_t M, int64_t K, bool up) {
    char* at = static_cast<char*>(buffer.data_ptr());
    const size_t n = static_cast<size_t>(M) * bitnet_ckpt_pad(K);
    gq = reinterpret_cast<int8_t*>(at);
    gs = reinterpret_cast<float*>(at + n);
    if (!up) return;
    at += half(M, K);
    uq = reinterpret_cast<int8_t*>(at);
    us = reinterpret_cast<float*>(at + n);
  }
};

Tensor gate_forward(const Tensor& gate, const Tensor& up, int64_t act, const Tensor& buffer) {
  const Tensor g = strided_rows(gate), u = up.defined() ? strided_rows(up) : Tensor();
  const int64_t M = g.size(0), K = g.size(1);
  Tensor y = at::empty(gate.sizes(), gate.options());
  if (M > 0) {
    const GateCodes c = buffer.defined() ? GateCodes(buffer, M, K, up.defined()) : GateCodes();
    On on(g);
    check(bitnet_gate_fwd(static_cast<bitnet_act>(act), bf16(g), row_stride(g), bf16(u), row_stride(u), M, K, bf16(y),
                          c.gq, c.gs, c.uq, c.us, on.stream));
  }
  return y;
}

struct GateFn : torch::autograd::Function<GateFn> {
  static Tensor forward(AutogradContext* ctx, const Tensor& gate, const optional<Tensor>& up, int64_t act,
                        bool checkpoint) {
    const Tensor u = up.value_or(Tensor());
    Tensor buffer;
    if (checkpoint) {
      const int64_t K = gate.size(-1), M = gate.numel() / K;
      buffer = scratch(GateCodes::half(M, K) * (u.defined() ? 2 : 1), gate);
      ctx->save_for_backward({buffer});
    } else {
      ctx->save_for_backward({gate, u});
    }
    ctx->saved_data["act"] = act;
    ctx->saved_data["checkpoint"] = checkpoint;
    ctx->saved_data["up"] = u.defined();
    return gate_forward(gate, u, act, buffer);
  }

  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    check_backward();
    const variable_list saved = ctx->get_saved_variables();
    const bool checkpoint = ctx->saved_data["checkpoint"].toBool(), gated = ctx->saved_data["up"].toBool();
    const auto act = static_cast<bitnet_act>(ctx->saved_data["act"].toInt());
    const auto shape = grads[0].sizes();
    const Tensor dY = rows(grads[0].to(at::kBFloat16));
    const int64_t M = dY.size(0), K = dY.size(1);
    Tensor dgate = at::empty(shape, dY.options()), dup = gated ? at::empty(shape, dY.options()) : Tensor();
    if (M > 0) {
      Tensor g, u;
      GateCodes c;
      if (checkpoint) {
        c = GateCodes(saved[0], M, K, gated);
      } else {
        g = strided_rows(saved[0]);
        if (gated) u = strided_rows(saved[1]);
      }
      On on(dY);
      check(bitnet_gate_bwd(act, bf16(dY), bf16(g), row_stride(g), bf16(u), row_stride(u), c.gq, c.gs, c.uq, c.us, M, K,
                            bf16(dgate), K, bf16(dup), K, on.stream));
    }
    return {dgate, dup, Tensor(), Tensor()};
  }
};

Tensor gated_activation(const Tensor& gate, const optional<Tensor>& up, int64_t act, bool checkpoint) {
  const Tensor u = up.value_or(Tensor());
  check_eager("gated_activation", {&gate, &u});
  TORCH_CHECK_TYPE(gate.scalar_type() == at::kBFloat16 && (!u.defined() || u.scalar_type() == at::kBFloat16),
                   "gated_activation expects bf16 activations");
  TORCH_CHECK_VALUE(!u.defined() || u.sizes() == gate.sizes(), "up: expected shape ", gate.sizes(), ", got ",
                    u.defined() ? u.sizes() : gate.sizes());
  check_activation("gated_activation", gate);
  TORCH_CHECK_VALUE(!u.defined() || u.device() == gate.device(), "gate and up: must be GPU tensors of one device");
  if (wants_grad({&gate, &u})) return GateFn::apply(gate, up, act, checkpoint);
  return gate_forward(gate, u, act, Tensor());
}

// --- the TTQ layer with an 8-bit checkpoint of its input --------------------------------

struct TtqFn : torch::autograd::Function<TtqFn> {
  // keep: dW or the scales' gradients are wanted, which alone read x
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const Tensor& weight, const Tensor& params, bool keep) {
    const Tensor x2 = aligned(rows(x)), w = aligned(weight), p = params.to(at::kFloat).contiguous();
    const int64_t M = x2.size(0), K = x2.size(1), N = w.size(0), Kp = bitnet_k_pad(K);
    std::vector<int64_t> shape = x.sizes().vec();
    shape.back() = N;
    Tensor y = at::empty(shape, x.options());
    ctx->saved_data["x"] = x.sizes();
    ctx->saved_data["wt"] = static_cast<int64_t>(weight.scalar_type());
    ctx->saved_data["n"] = N;
    if (M == 0) return y;
    const Tensor codes_w = at::empty({N, Kp / 4}, x.options().dtype(at::kByte)), wt = at::empty({N, Kp}, x.options());
    const size_t bytes = ttq_fwd_ckpt_workspace_bytes(M, N, K);
    const Tensor ws = scratch(bytes, x);
    Tensor codes, scales;
    if (keep) std::tie(codes, scales) = empty_codes(M, K, x2);
    On on(x2);
    check(ttq_quantize(ptr(w), code(w.scalar_type()), N, K, f32(p), static_cast<uint8_t*>(ptr(codes_w)), bf16(wt),
                       on.stream));
    check(ttq_fwd_ckpt(bf16(x2), bf16(wt), M, N, K, bf16(y), i8(codes), f32(scales), ptr(ws), bytes, on.stream));
    ctx->save_for_backward({codes, scales, wt, codes_w});
    return y;
  }

  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    check_backward();
    const std::vector<int64_t> shape = ctx->saved_data["x"].toIntVector();
    const auto wdt = static_cast<at::ScalarType>(ctx->saved_data["wt"].toInt());
    const int64_t K = shape.back(), N = ctx->saved_data["n"].toInt();
    const bool need_x = ctx->needs_input_grad(0), need_w = ctx->needs_input_grad(1), need_p = ctx->needs_input_grad(2);
    Tensor dX, dW, dp;
    if (grads[0].numel() == 0) {  // no rows
      const auto o = grads[0].options();
      if (need_x) dX = at::empty(shape, o.dtype(at::kBFloat16));
      if (need_w) dW = at::zeros({N, K}, o.dtype(wdt));
      if (need_p) dp = at::zeros({3}, o.dtype(at::kFloat));
      return {dX, dW, dp, Tensor()};
    }
    const variable_list saved = ctx->get_saved_variables();
    const Tensor &codes = saved[0], &scales = saved[1], &wt = saved[2], &codes_w = saved[3];
    const Tensor dY = aligned(rows(grads[0].to(at::kBFloat16)));
    const int64_t M = dY.size(0);
    if (need_x) dX = at::empty(shape, dY.options());
    // the scales' gradients come from dW's epilogue; the threshold has none
    if (need_w || need_p) dW = at::empty({N, K}, dY.options().dtype(wdt));
    if (need_p) dp = at::zeros({3}, dY.options().dtype(at::kFloat));
    const size_t bytes = ttq_bwd_ckpt_workspace_bytes(M, N, K);
    const Tensor ws = scratch(bytes, dY);
    On on(dY);
    check(ttq_bwd_ckpt(bf16(dY), i8(codes), f32(scales), bf16(wt), static_cast<uint8_t*>(ptr(codes_w)), M, N, K, bf16(dX),
                       ptr(dW), code(wdt), dp.defined() ? f32(dp) + 1 : nullptr, ptr(ws), bytes, on.stream));
    return {dX, need_w ? dW : Tensor(), dp, Tensor()};
  }
};

Tensor ttq_linear_checkpoint(const Tensor& x, const Tensor& weight, const Tensor& params) {
  check_eager("ttq_linear", {&x, &weight, &params});
  TORCH_CHECK_TYPE(x.scalar_type() == at::kBFloat16, "TTQ expects bf16 activations");
  TORCH_CHECK_TYPE(is_value(weight.scalar_type()), "weight: expected bf16 or float32, got ", weight.scalar_type());
  check_activation("ttq_linear", x);
  TORCH_CHECK_VALUE(weight.dim() == 2 && weight.size(1) == x.size(-1) && weight.size(0) >= 1,
                    "weight: expected [out_features, ", x.size(-1), "], got ", weight.sizes());
  TORCH_CHECK_VALUE(params.numel() == 3 && params.dim() == 1, "params: expected shape [3], got ", params.sizes());
  TORCH_CHECK_VALUE(weight.device() == x.device() && params.device() == x.device(),
                    "x, weight and params: must be GPU tensors of one device");
  return TtqFn::apply(x, weight, params, wants_grad({&weight, &params}));
}

// --- linear layer with cross entropy -------------------------------------------------

struct Xent {
  Tensor h, w, t, loss, lse, total;
  Xent(const Tensor& h_, const Tensor& w_, const Tensor& t_, int64_t ignore, int64_t reduce)
      : h(aligned(h_)), w(aligned(w_.to(at::kBFloat16))), t(t_.contiguous()) {
    const int64_t T = h.size(0), D = h.size(1), V = w.size(0);
    const auto o = h.options().dtype(at::kFloat);
    loss = at::empty({T}, o);
    lse = at::empty({T}, o);
    if (reduce != BITNET_REDUCE_NONE) total = at::empty({}, o);
    const size_t bytes = bitnet_xent_fwd_workspace_bytes(T, V, D);
    const Tensor ws = scratch(bytes, h);
    On on(h);
    check(bitnet_xent_fwd(bf16(h), bf16(w), static_cast<const int64_t*>(ptr(t)), ignore, T, V, D, f32(loss), f32(lse),
                          f32(total), static_cast<bitnet_reduce>(reduce), ptr(ws), bytes, on.stream));
  }
  const Tensor& result() const { return total.defined() ? total : loss; }
};

struct XentFn : torch::autograd::Function<XentFn> {
  static Tensor forward(AutogradContext* ctx, const Tensor& h, const Tensor& w, const Tensor& t, int64_t ignore,
                        int64_t reduce) {
    const Xent x(h, w, t, ignore, reduce);
    ctx->save_for_backward({x.h, x.w, x.t, x.lse});
    ctx->saved_data["ignore"] = ignore;
    ctx->saved_data["reduce"] = reduce;
    ctx->saved_data["wt"] = static_cast<int64_t>(w.scalar_type());
    return x.result();
  }

  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    check_backward();
    const variable_list saved = ctx->get_saved_variables();
    const Tensor &h = saved[0], &w = saved[1], &t = saved[2], &lse = saved[3];
    const auto reduce = static_cast<bitnet_reduce>(ctx->saved_data["reduce"].toInt());
    const auto wt = static_cast<at::ScalarType>(ctx->saved_data["wt"].toInt());
    const int64_t T = h.size(0), D = h.size(1), V = w.size(0);
    Tensor dh, dw;
    if (ctx->needs_input_grad(0)) dh = at::empty({T, D}, h.options());
    if (ctx->needs_input_grad(1)) dw = at::empty({V, D}, h.options().dtype(wt));
    const Tensor c = grads[0].to(at::kFloat).contiguous();
    const size_t bytes = bitnet_xent_bwd_workspace_bytes(T, V, D);
    const Tensor ws = scratch(bytes, h);
    On on(h);
    check(bitnet_xent_bwd(bf16(h), bf16(w), static_cast<const int64_t*>(ptr(t)), ctx->saved_data["ignore"].toInt(),
                          f32(lse), f32(c), reduce, T, V, D, bf16(dh), ptr(dw), code(wt), ptr(ws), bytes, on.stream));
    return {dh, dw, Tensor(), Tensor(), Tensor()};
  }
};

Tensor linear_cross_entropy(const Tensor& hidden, const Tensor& weight, const Tensor& targets, int64_t ignore,
                            int64_t reduce) {
  check_eager("linear_cross_entropy", {&hidden, &weight, &targets});
  TORCH_CHECK_TYPE(hidden.scalar_type() == at::kBFloat16, "linear_cross_entropy expects bf16 hidden states, got ",
                   hidden.scalar_type());
  TORCH_CHECK_TYPE(is_value(weight.scalar_type()), "weight: expected bf16 or float32, got ", weight.scalar_type());
  TORCH_CHECK_TYPE(targets.scalar_type() == at::kLong, "targets: expected int64, got ", targets.scalar_type());
  TORCH_CHECK_VALUE(hidden.dim() >= 1 && weight.dim() == 2 && weight.size(1) == hidden.size(-1) && weight.numel() > 0,
                    "weight: expected [vocabulary, features] for hidden states ", hidden.sizes(), ", got ",
                    weight.sizes());
  TORCH_CHECK_VALUE(targets.sizes() == hidden.sizes().slice(0, hidden.dim() - 1), "targets: expected shape ",
                    hidden.sizes().slice(0, hidden.dim() - 1), ", got ", targets.sizes());
  TORCH_CHECK_VALUE(hidden.is_cuda() && weight.device() == hidden.device() && targets.device() == hidden.device(),
                    "hidden, weight and targets: must be GPU tensors of one device");
  const Tensor h = hidden.dim() == 2 ? hidden : hidden.reshape({-1, hidden.size(-1)});
  const Tensor t = targets.reshape({-1});
  Tensor out;
  if (t.size(0) == 0) {  // no rows: zeros that still depend on both inputs
    out = h.sum(at::kFloat) + weight.slice(0, 0, 0).sum(at::kFloat);
    return reduce == BITNET_REDUCE_NONE ? out + at::zeros(targets.sizes(), out.options()) : out;
  }
  if (wants_grad({&hidden, &weight})) out = XentFn::apply(h, weight, t, ignore, reduce);
  else out = Xent(h, weight, t, ignore, reduce).result();
  return reduce == BITNET_REDUCE_NONE && targets.dim() != 1 ? out.reshape(targets.sizes()) : out;
}

}  // namespace

PYBIND11_MODULE(_bitnet_ops, m) {
  const auto free_gil = py::call_guard<py::gil_scoped_release>();
  m.def("layer_norm", &layer_norm, free_gil);
  m.def("compress", &compress, free_gil);
  m.def("decompress", &decompress, free_gil);
  m.def("gated_activation", &gated_activation, free_gil);
  m.def("ttq_linear_checkpoint", &ttq_linear_checkpoint, free_gil);
  m.def("linear_cross_entropy", &linear_cross_entropy, free_gil);
}
