// The operators around the ternary linear layers as torch autograd functions
// over the C ABI (include/bitnet.h): layer norm, 8-bit activation checkpoints,
// the gated activation, the TTQ layer with its input kept in 8 bits, the
// linear layer with cross entropy, the root-mean-square norm with 8-bit rows,
// the gated pair of ternary projections and the linear layer in 8-bit integers.
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

// --- 8-bit rows ----------------------------------------------------------------------

// Rows of 8-bit codes with a scale each, as the functions take them: codes [M, Kp],
// scales [M], and a carrier, a bf16 tensor of the shape [..., K] that the rows
// stand for, whose strides are 0 (it holds no values, only the shape and the
// place in the autograd graph that gradients of the rows' values go to).
Tensor make_carrier(at::IntArrayRef shape, const Tensor& like) {
  return at::empty_strided(shape, std::vector<int64_t>(shape.size(), 0), like.options().dtype(at::kBFloat16));
}

void check_rows(const char* what, const Tensor& carrier, const Tensor& codes, const Tensor& scales) {
  TORCH_CHECK_TYPE(codes.scalar_type() == at::kChar && scales.scalar_type() == at::kFloat &&
                       carrier.scalar_type() == at::kBFloat16,
                   what, ": 8-bit rows have int8 codes and float32 scales, got ", codes.scalar_type(), " and ",
                   scales.scalar_type());
  check_activation(what, carrier);
  const int64_t K = carrier.size(-1), M = carrier.numel() / K;
  TORCH_CHECK_VALUE(codes.dim() == 2 && codes.size(0) == M && codes.size(1) == bitnet_k_pad(K) && scales.dim() == 1 &&
                        scales.size(0) == M,
                    what, ": not the 8-bit rows of ", carrier.sizes(), ": codes ", codes.sizes(), " and scales ",
                    scales.sizes());
  TORCH_CHECK_VALUE(codes.device() == carrier.device() && scales.device() == carrier.device(), what,
                    ": codes and scales must be on ", carrier.device());
}

Tensor unpack_rows(const Tensor& carrier, const Tensor& codes, const Tensor& scales) {
  const Tensor q = aligned(codes), s = scales.contiguous();
  Tensor x = at::empty(carrier.sizes(), carrier.options());
  if (x.numel() > 0) {
    On on(q);
    check(bitnet_rows_unpack(i8(q), f32(s), q.size(0), carrier.size(-1), bf16(x), on.stream));
  }
  return x;
}

struct UnpackRowsFn : torch::autograd::Function<UnpackRowsFn> {
  static Tensor forward(AutogradContext*, const Tensor& carrier, const Tensor& codes, const Tensor& scales) {
    return unpack_rows(carrier, codes, scales);
  }
  static variable_list backward(AutogradContext*, const variable_list& grads) {
    check_backward();
    return {grads[0], Tensor(), Tensor()};
  }
};

Tensor rows_values(const Tensor& carrier, const Tensor& codes, const Tensor& scales) {
  check_eager("dequantize", {&carrier, &codes, &scales});
  check_rows("dequantize", carrier, codes, scales);
  return wants_grad({&carrier}) ? UnpackRowsFn::apply(carrier, codes, scales) : unpack_rows(carrier, codes, scales);
}

// x of a layer as 8-bit rows: those given, or made of bf16 activations.
struct Rows {
  Tensor q, s, x2;  // x2: activations that are still to be quantized into q and s
  int64_t M, K;
  bool direct = false;  // x2 goes to the kernel as it is; there are no q and s
  // may_direct: where the product takes so few rows itself.
  Rows(const Tensor& x, const Tensor& codes, const Tensor& scales, bool may_direct = false) : K(x.size(-1)) {
    M = x.numel() / K;
    if (codes.defined()) {
      q = aligned(codes);
      s = aligned(scales);
      return;
    }
    direct = may_direct && M <= bitnet_rows_direct(K);
    x2 = direct ? rows(x) : aligned(rows(x));
    if (direct) return;
    q = at::empty({M, bitnet_k_pad(K)}, x.options().dtype(at::kChar));
    s = at::empty({M}, x.options().dtype(at::kFloat));
  }
  void quantize(void* stream) const {
    if (x2.defined() && !direct) check(bitnet_rows_quant(bf16(x2), BITNET_BF16, M, K, i8(q), f32(s), stream));
  }
};

void check_layer_input(const char* what, const Tensor& x, const Tensor& codes, const Tensor& scales) {
  if (codes.defined() || scales.defined()) {
    TORCH_CHECK_VALUE(codes.defined() && scales.defined(), what, ": codes and scales: both needed");
    check_rows(what, x, codes, scales);
  } else {
    TORCH_CHECK_TYPE(x.scalar_type() == at::kBFloat16, what, " expects bf16 activations, got ", x.scalar_type());
    check_activation(what, x);
  }
}

std::vector<int64_t> with_last(at::IntArrayRef shape, int64_t n) {
  std::vector<int64_t> s = shape.vec();
  s.back() = n;
  return s;
}

// --- root-mean-square norm -------------------------------------------------------------

struct Rms {
  Tensor x2, r2, w, h, y, q, s, rstd;
  int64_t M, K;
  // out undefined: 8-bit rows (y is their carrier)
  Rms(const Tensor& x, const Tensor& weight, const Tensor& residual, double eps, optional<at::ScalarType> out, bool keep)
      : x2(rows(x)), M(x2.size(0)), K(x2.size(1)) {
    if (weight.defined()) w = weight.contiguous();
    if (residual.defined()) {
      r2 = rows(residual);
      h = at::empty(x.sizes(), residual.options());
    }
    const auto o = x.options();
    if (out.has_value()) {
      y = at::empty(x.sizes(), o.dtype(*out));
    } else {
      y = make_carrier(x.sizes(), x);
      q = at::empty({M, bitnet_k_pad(K)}, o.dtype(at::kChar));
      s = at::empty({M}, o.dtype(at::kFloat));
    }
    if (keep) rstd = at::empty({M}, o.dtype(at::kFloat));
    if (M == 0) return;
    const bitnet_dtype xd = code(x2.scalar_type()), hd = r2.defined() ? code(r2.scalar_type()) : xd;
    On on(x2);
    check(bitnet_rmsnorm_fwd(ptr(x2), xd, ptr(r2), hd, ptr(w), w.defined() ? code(w.scalar_type()) : BITNET_F32, M, K,
                             static_cast<float>(eps), ptr(h), out.has_value() ? ptr(y) : nullptr, code(y.scalar_type()),
                             i8(q), f32(s), f32(rstd), on.stream));
  }
};

// Outputs: y (or the rows' carrier), codes and scales (undefined without), h
// (undefined without a residual).
struct RmsNormFn : torch::autograd::Function<RmsNormFn> {
  static variable_list forward(AutogradContext* ctx, const Tensor& x, const optional<Tensor>& weight,
                               const optional<Tensor>& residual, double eps, bool quantize, at::ScalarType out) {
    const Tensor r = residual.value_or(Tensor());
    const Rms n(x, weight.value_or(Tensor()), r, eps, quantize ? optional<at::ScalarType>() : out, true);
    ctx->save_for_backward({r.defined() ? n.h : n.x2, n.w, n.rstd});
    ctx->set_materialize_grads(false);
    ctx->saved_data["shape"] = x.sizes();
    ctx->saved_data["x"] = static_cast<int64_t>(x.scalar_type());
    ctx->saved_data["y"] = static_cast<int64_t>(n.y.scalar_type());
    ctx->saved_data["quantize"] = quantize;
    ctx->saved_data["w"] = weight.has_value();
    ctx->saved_data["r"] = residual.has_value();
    variable_list res{n.y};
    if (quantize) {
      ctx->mark_non_differentiable({n.q, n.s});
      res.push_back(n.q);
      res.push_back(n.s);
    }
    if (r.defined()) res.push_back(n.h);
    return res;
  }

  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    check_backward();
    const variable_list saved = ctx->get_saved_variables();
    const Tensor &h = saved[0], &w = saved[1], &rstd = saved[2];
    const std::vector<int64_t> shape = ctx->saved_data["shape"].toIntVector();
    const auto xt = static_cast<at::ScalarType>(ctx->saved_data["x"].toInt());
    const auto yt = static_cast<at::ScalarType>(ctx->saved_data["y"].toInt());
    const bool quantize = ctx->saved_data["quantize"].toBool();
    const bool has_w = ctx->saved_data["w"].toBool(), has_r = ctx->saved_data["r"].toBool();
    const bool need_x = ctx->needs_input_grad(0), need_w = has_w && ctx->needs_input_grad(1);
    const bool need_r = has_r && ctx->needs_input_grad(1 + has_w);
    const auto ht = h.scalar_type();
    const int64_t K = shape.back(), M = rstd.size(0);
    Tensor dH = has_r ? grads[quantize ? 3 : 1] : Tensor();
    Tensor dx, dr, dw;
    const auto ho = h.options();
    if (!grads[0].defined() || M == 0) {  // the norm's output was not used, or has no rows
      if (need_w) dw = at::zeros({K}, w.options());
      if (!dH.defined() && M == 0) dH = at::zeros(shape, ho);
      if (dH.defined()) {
        if (need_x) dx = dH.to(xt);
        if (need_r) dr = dH.to(ht);
      }
      return {dx, dw, dr, Tensor(), Tensor(), Tensor()};
    }
    const Tensor dY = rows(grads[0].to(yt));
    if (dH.defined()) dH = rows(dH.to(ht));
    // one gradient for both where they are of one type
    const bool split = xt != ht;
    if ((need_x && !split) || need_r) dr = at::empty(shape, ho);
    if (need_x) dx = split ? at::empty(shape, ho.dtype(xt)) : dr;
    Tensor ws;
    size_t bytes = 0;
    if (need_w) {
      dw = at::empty({K}, w.options());
      bytes = bitnet_rmsnorm_workspace_bytes(M, K);
      ws = scratch(bytes, dY);
    }
    On on(dY);
    check(bitnet_rmsnorm_bwd(ptr(dY), code(yt), ptr(dH), ptr(h), code(ht), ptr(w),
                             w.defined() ? code(w.scalar_type()) : BITNET_F32, f32(rstd), M, K, ptr(dr),
                             split && need_x ? bf16(dx) : nullptr, ptr(dw), ptr(ws), bytes, on.stream));
    return {dx, dw, need_r ? dr : Tensor(), Tensor(), Tensor(), Tensor()};
  }
};

// (y or the rows' carrier, codes, scales, h), those that there are.
std::tuple<Tensor, Tensor, Tensor, Tensor> rms_norm(const Tensor& x, const optional<Tensor>& weight,
                                                    const optional<Tensor>& residual, double eps, bool quantize,
                                                    at::ScalarType out) {
  const Tensor w = weight.value_or(Tensor()), r = residual.value_or(Tensor());
  check_eager("rms_norm", {&x, &w, &r});
  TORCH_CHECK_TYPE(is_value(x.scalar_type()), "rms_norm expects bf16 or float32 activations, got ", x.scalar_type());
  TORCH_CHECK_TYPE(is_value(out), "out_dtype: expected bfloat16 or float32, got ", out);
  check_activation("rms_norm", x);
  if (w.defined()) {
    TORCH_CHECK_TYPE(is_value(w.scalar_type()), "weight: expected bf16 or float32, got ", w.scalar_type());
    TORCH_CHECK_VALUE(w.dim() == 1 && w.size(0) == x.size(-1), "weight: expected shape [", x.size(-1), "], got ",
                      w.sizes());
    TORCH_CHECK_VALUE(w.device() == x.device(), "weight: on ", w.device(), ", expected ", x.device());
  }
  if (r.defined()) {
    TORCH_CHECK_TYPE(is_value(r.scalar_type()), "residual: expected bf16 or float32, got ", r.scalar_type());
    TORCH_CHECK_TYPE(x.scalar_type() == at::kBFloat16 || x.scalar_type() == r.scalar_type(),
                     "x: expected bf16 or the residual's dtype, got ", x.scalar_type());
    TORCH_CHECK_VALUE(r.sizes() == x.sizes(), "residual: expected shape ", x.sizes(), ", got ", r.sizes());
    TORCH_CHECK_VALUE(r.device() == x.device(), "residual: on ", r.device(), ", expected ", x.device());
  }
  if (wants_grad({&x, &w, &r})) {
    const variable_list o = RmsNormFn::apply(x, weight, residual, eps, quantize, out);
    if (quantize) return {o[0], o[1], o[2], r.defined() ? o[3] : Tensor()};
    return {o[0], Tensor(), Tensor(), r.defined() ? o[1] : Tensor()};
  }
  const Rms n(x, w, r, eps, quantize ? optional<at::ScalarType>() : out, false);
  return {n.y, n.q, n.s, n.h};
}

// --- the gated pair of ternary projections ------------------------------------------------

// Both weights' codes below each other and both scales; x is quantized with
// them where it still is to be.
struct GatedState {
  Tensor packed, gamma;
  GatedState(const Rows& x, const Tensor& w_gate, const Tensor& w_up) {
    const Tensor wg = aligned(w_gate), wu = aligned(w_up);
    const int64_t N = wg.size(0), K = x.K, row = bitnet_k_pad(K) / 4;
    packed = at::empty({2 * N, row}, wg.options().dtype(at::kByte));
    gamma = at::empty({2}, wg.options().dtype(at::kFloat));
    const size_t bytes = bitnet_ternarize_workspace_bytes(N, K);
    const Tensor ws = scratch(bytes, wg);
    const bool rows = x.x2.defined() && x.M > 0;
    On on(wg);
    check(bitnet_quantize2(ptr(wg), ptr(wu), code(wg.scalar_type()), N, K, rows ? bf16(x.x2) : nullptr, x.M,
                           static_cast<uint8_t*>(ptr(packed)), f32(gamma), i8(x.q), f32(x.s), ptr(ws), bytes,
                           on.stream));
  }
};

Tensor gated_forward(const Rows& x, at::IntArrayRef shape, const Tensor& packed, const Tensor& gamma, int64_t act,
                     const Tensor& slopes) {
  const int64_t N = packed.size(0) / 2;
  Tensor y = at::empty(with_last(shape, N), packed.options().dtype(at::kBFloat16));
  if (x.M == 0) return y;
  const size_t bytes = bitnet_gated_fwd_workspace_bytes(x.M, N, x.K);
  const Tensor ws = scratch(bytes, packed);
  On on(packed);
  check(bitnet_gated_fwd(static_cast<bitnet_act>(act), x.direct ? bf16(x.x2) : nullptr, i8(x.q), f32(x.s),
                         static_cast<uint8_t*>(ptr(packed)), f32(gamma), x.M, N, x.K, bf16(y), ptr(slopes), bytes ? ptr(ws) : nullptr, bytes, on.stream));
  return y;
}

Tensor empty_slopes(int64_t M, int64_t N, const Tensor& like) {
  return scratch(bitnet_gated_slopes_bytes(M, N), like);
}

struct GatedGrads {
  Tensor dx, dwg, dwu;
};
GatedGrads gated_backward(const Tensor& grad, const Tensor& slopes, const Tensor& q, const Tensor& s,
                          const Tensor& packed, const Tensor& gamma, at::IntArrayRef shape, bool need_x,
                          bool need_w, at::ScalarType wt) {
  GatedGrads r;
  const int64_t N = packed.size(0) / 2, K = shape.back(), M = q.size(0);
  const Tensor dY = rows(grad.to(at::kBFloat16));
  if (need_x) r.dx = at::empty(shape, dY.options());
  if (need_w) {
    const auto o = dY.options().dtype(wt);
    r.dwg = M > 0 ? at::empty({N, K}, o) : at::zeros({N, K}, o);
    r.dwu = M > 0 ? at::empty({N, K}, o) : at::zeros({N, K}, o);
  }
  if (M == 0 || (!need_x && !need_w)) return r;
  const size_t bytes = bitnet_gated_bwd_workspace_bytes(M, N, K);
  const Tensor ws = scratch(bytes, dY);
  On on(dY);
  check(bitnet_gated_bwd(bf16(dY), ptr(slopes), i8(q), f32(s),
                         static_cast<uint8_t*>(ptr(packed)), f32(gamma), M, N, K, bf16(r.dx), ptr(r.dwg), ptr(r.dwu),
                         code(wt), ptr(ws), bytes, on.stream));
  return r;
}

struct GatedFn : torch::autograd::Function<GatedFn> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const optional<Tensor>& codes,
                        const optional<Tensor>& scales, const Tensor& w_gate, const Tensor& w_up, int64_t act) {
    const Rows r(x, codes.value_or(Tensor()), scales.value_or(Tensor()));
    const GatedState st(r, w_gate, w_up);
    const Tensor slopes = empty_slopes(r.M, w_gate.size(0), r.q);
    Tensor y = gated_forward(r, x.sizes(), st.packed, st.gamma, act, slopes);
    ctx->save_for_backward({slopes, r.q, r.s, st.packed, st.gamma});
    ctx->saved_data["shape"] = x.sizes();
    ctx->saved_data["wt"] = static_cast<int64_t>(w_gate.scalar_type());
    ctx->saved_data["at"] = static_cast<int64_t>(codes.has_value() ? 3 : 1);  // the gate weight's place among the tensors
    return y;
  }
  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    check_backward();
    const variable_list v = ctx->get_saved_variables();
    const int64_t at = ctx->saved_data["at"].toInt();
    const bool need_g = ctx->needs_input_grad(at), need_u = ctx->needs_input_grad(at + 1);
    const GatedGrads r = gated_backward(grads[0], v[0], v[1], v[2], v[3], v[4], ctx->saved_data["shape"].toIntVector(),
                                        ctx->needs_input_grad(0), need_g || need_u,
                                        static_cast<at::ScalarType>(ctx->saved_data["wt"].toInt()));
    return {r.dx, Tensor(), Tensor(), need_g ? r.dwg : Tensor(), need_u ? r.dwu : Tensor(), Tensor()};
  }
};

Tensor gated_bitlinear(const Tensor& x, const optional<Tensor>& codes, const optional<Tensor>& scales,
                       const Tensor& w_gate, const Tensor& w_up, int64_t act) {
  const Tensor q = codes.value_or(Tensor()), s = scales.value_or(Tensor());
  check_eager("gated_bitlinear", {&x, &q, &s, &w_gate, &w_up});
  check_layer_input("gated_bitlinear", x, q, s);
  TORCH_CHECK_TYPE(is_value(w_gate.scalar_type()) && w_up.scalar_type() == w_gate.scalar_type(),
                   "w_gate and w_up: expected bf16 or float32 and one dtype, got ", w_gate.scalar_type(), " and ",
                   w_up.scalar_type());
  TORCH_CHECK_VALUE(w_gate.dim() == 2 && w_gate.size(1) == x.size(-1) && w_gate.size(0) >= 1 &&
                        w_up.sizes() == w_gate.sizes(),
                    "w_gate and w_up: expected [out_features, ", x.size(-1), "] both, got ", w_gate.sizes(), " and ",
                    w_up.sizes());
  TORCH_CHECK_VALUE(w_gate.device() == x.device() && w_up.device() == x.device(),
                    "x, w_gate and w_up: must be GPU tensors of one device");
  if (wants_grad({&x, &w_gate, &w_up})) return GatedFn::apply(x, codes, scales, w_gate, w_up, act);
  const Rows r(x, q, s);
  const GatedState st(r, w_gate, w_up);
  return gated_forward(r, x.sizes(), st.packed, st.gamma, act, Tensor());
}

// The same from the stored state; gradients of x alone.
struct GatedFrozenFn : torch::autograd::Function<GatedFrozenFn> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const optional<Tensor>& codes,
                        const optional<Tensor>& scales, const Tensor& packed, const Tensor& gamma, int64_t act) {
    const Rows r(x, codes.value_or(Tensor()), scales.value_or(Tensor()), true);
    const Tensor slopes = empty_slopes(r.M, packed.size(0) / 2, packed);
    if (r.M > 0) {
      On on(packed);
      r.quantize(on.stream);
    }
    Tensor y = gated_forward(r, x.sizes(), packed, gamma, act, slopes);
    ctx->save_for_backward({slopes, packed, gamma});
    ctx->saved_data["m"] = r.M;
    ctx->saved_data["shape"] = x.sizes();
    return y;
  }
  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    check_backward();
    const variable_list v = ctx->get_saved_variables();
    const std::vector<int64_t> shape = ctx->saved_data["shape"].toIntVector();
    const Tensor &slopes = v[0], &packed = v[1], &gamma = v[2];
    const Tensor dY = rows(grads[0].to(at::kBFloat16));
    const int64_t N = packed.size(0) / 2, K = shape.back(), M = ctx->saved_data["m"].toInt();
    const Tensor dx = at::empty(shape, dY.options());
    if (M > 0) {
      const size_t bytes = bitnet_gated_bwd_workspace_bytes(M, N, K);
      const Tensor ws = scratch(bytes, dY);
      On on(dY);
      check(bitnet_gated_bwd(bf16(dY), ptr(slopes), nullptr, nullptr,
                             static_cast<uint8_t*>(ptr(packed)), f32(gamma), M, N, K, bf16(dx), nullptr, nullptr,
                             BITNET_BF16, ptr(ws), bytes, on.stream));
    }
    return {dx, Tensor(), Tensor(), Tensor(), Tensor(), Tensor()};
  }
};

Tensor gated_bitlinear_inference(const Tensor& x, const optional<Tensor>& codes, const optional<Tensor>& scales,
                                 const Tensor& w_packed, const Tensor& gamma_, int64_t in_features, int64_t act) {
  const Tensor q = codes.value_or(Tensor()), s = scales.value_or(Tensor());
  check_eager("gated_bitlinear", {&x, &q, &s, &w_packed, &gamma_});
  check_layer_input("gated_bitlinear", x, q, s);
  TORCH_CHECK_VALUE(x.size(-1) == in_features, "x: expected a last dimension of ", in_features, ", got ", x.sizes());
  TORCH_CHECK_TYPE(w_packed.scalar_type() == at::kByte && gamma_.scalar_type() == at::kFloat,
                   "w_packed: expected uint8 and gamma float32, got ", w_packed.scalar_type(), " and ",
                   gamma_.scalar_type());
  TORCH_CHECK_VALUE(w_packed.dim() == 2 && w_packed.size(0) >= 2 && w_packed.size(0) % 2 == 0 &&
                        w_packed.size(1) == bitnet_k_pad(in_features) / 4 && gamma_.dim() == 1 && gamma_.size(0) == 2,
                    "w_packed: expected [2 out_features, ", bitnet_k_pad(in_features) / 4, "] and gamma [2], got ",
                    w_packed.sizes(), " and ", gamma_.sizes());
  TORCH_CHECK_VALUE(w_packed.device() == x.device() && gamma_.device() == x.device(),
                    "x, w_packed and gamma: must be GPU tensors of one device");
  const Tensor packed = aligned(w_packed), gamma = gamma_.contiguous();
  if (wants_grad({&x})) return GatedFrozenFn::apply(x, codes, scales, packed, gamma, act);
  const Rows r(x, q, s, true);
  if (r.M > 0) {
    On on(packed);
    r.quantize(on.stream);
  }
  return gated_forward(r, x.sizes(), packed, gamma, act, Tensor());
}

// --- linear layer in 8-bit integers -----------------------------------------------------------

// The weight's rows as int8 with a scale each, and those of x that are still to be made.
std::pair<Tensor, Tensor> int8_weight(const Tensor& weight, const Rows* x) {
  const Tensor w = weight.contiguous();
  const int64_t N = w.size(0), K = w.size(1), M = x && x->x2.defined() ? x->M : 0;
  std::pair<Tensor, Tensor> r{at::empty({N, bitnet_k_pad(K)}, w.options().dtype(at::kChar)),
                              at::empty({N}, w.options().dtype(at::kFloat))};
  On on(w);
  check(bitnet_rows_quant2(M ? bf16(x->x2) : nullptr, M, M ? i8(x->q) : nullptr, M ? f32(x->s) : nullptr, ptr(w),
                           code(w.scalar_type()), N, i8(r.first), f32(r.second), K, on.stream));
  return r;
}

Tensor int8_forward(const Rows& x, at::IntArrayRef shape, const Tensor& wq, const Tensor& sw, const Tensor& bias) {
  const int64_t N = wq.size(0);
  Tensor y = at::empty(with_last(shape, N), wq.options().dtype(at::kBFloat16));
  if (x.M == 0) return y;
  const Tensor b = bias.defined() ? aligned(bias.to(at::kBFloat16)) : Tensor();
  const size_t bytes = bitnet_int8_fwd_workspace_bytes(x.M, N, x.K);
  const Tensor ws = scratch(bytes, wq);
  On on(wq);
  check(bitnet_int8_fwd(x.direct ? bf16(x.x2) : nullptr, i8(x.q), f32(x.s), i8(wq), f32(sw), bf16(b), x.M, N, x.K, bf16(y), bytes ? ptr(ws) : nullptr,
                        bytes, on.stream));
  return y;
}

// Those that are wanted.
void int8_backward(const Tensor& grad, const Tensor& q, const Tensor& s, const Tensor& wq, const Tensor& sw,
                   at::IntArrayRef shape, Tensor* dx, Tensor* dw, at::ScalarType wt, Tensor* db, at::ScalarType bt) {
  const int64_t N = wq.size(0), K = shape.back();
  const Tensor dY = aligned(rows(grad.to(at::kBFloat16)));
  const int64_t M = dY.size(0);
  const auto o = dY.options();
  if (dx) *dx = at::empty(shape, o);
  if (M == 0) {
    if (dw) *dw = at::zeros({N, K}, o.dtype(wt));
    if (db) *db = at::zeros({N}, o.dtype(bt));
    return;
  }
  if (dw) *dw = at::empty({N, K}, o.dtype(wt));
  if (db) *db = at::empty({N}, o.dtype(bt));
  if (!dx && !dw && !db) return;
  const size_t bytes = bitnet_int8_bwd_workspace_bytes(M, N, K);
  const Tensor ws = scratch(bytes, dY);
  On on(dY);
  check(bitnet_int8_bwd(bf16(dY), dw ? i8(q) : nullptr, dw ? f32(s) : nullptr, dx ? i8(wq) : nullptr,
                        dx ? f32(sw) : nullptr, M, N, K, dx ? bf16(*dx) : nullptr, dw ? ptr(*dw) : nullptr, code(wt),
                        db ? ptr(*db) : nullptr, code(bt), ptr(ws), bytes, on.stream));
}

struct Int8Fn : torch::autograd::Function<Int8Fn> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const optional<Tensor>& codes,
                        const optional<Tensor>& scales, const Tensor& weight, const optional<Tensor>& bias) {
    const Rows r(x, codes.value_or(Tensor()), scales.value_or(Tensor()));
    const auto w = int8_weight(weight, &r);
    Tensor y = int8_forward(r, x.sizes(), w.first, w.second, bias.value_or(Tensor()));
    ctx->save_for_backward({r.q, r.s, w.first, w.second});
    ctx->saved_data["shape"] = x.sizes();
    ctx->saved_data["wt"] = static_cast<int64_t>(weight.scalar_type());
    ctx->saved_data["bt"] = static_cast<int64_t>(bias.has_value() ? bias->scalar_type() : at::kBFloat16);
    ctx->saved_data["b"] = bias.has_value();
    ctx->saved_data["at"] = static_cast<int64_t>(codes.has_value() ? 3 : 1);  // the weight's place among the tensors
    return y;
  }
  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    check_backward();
    const variable_list v = ctx->get_saved_variables();
    const int64_t at = ctx->saved_data["at"].toInt();
    const bool need_x = ctx->needs_input_grad(0), need_w = ctx->needs_input_grad(at);
    const bool need_b = ctx->saved_data["b"].toBool() && ctx->needs_input_grad(at + 1);
    Tensor dx, dw, db;
    int8_backward(grads[0], v[0], v[1], v[2], v[3], ctx->saved_data["shape"].toIntVector(), need_x ? &dx : nullptr,
                  need_w ? &dw : nullptr, static_cast<at::ScalarType>(ctx->saved_data["wt"].toInt()),
                  need_b ? &db : nullptr, static_cast<at::ScalarType>(ctx->saved_data["bt"].toInt()));
    return {dx, Tensor(), Tensor(), dw, db};
  }
};

// The same from the stored state; gradients of x and the bias.
struct Int8FrozenFn : torch::autograd::Function<Int8FrozenFn> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const optional<Tensor>& codes,
                        const optional<Tensor>& scales, const Tensor& wq, const Tensor& sw, const optional<Tensor>& bias) {
    const Rows r(x, codes.value_or(Tensor()), scales.value_or(Tensor()), true);
    if (r.M > 0) {
      On on(wq);
      r.quantize(on.stream);
    }
    Tensor y = int8_forward(r, x.sizes(), wq, sw, bias.value_or(Tensor()));
    ctx->save_for_backward({wq, sw});
    ctx->saved_data["shape"] = x.sizes();
    ctx->saved_data["bt"] = static_cast<int64_t>(bias.has_value() ? bias->scalar_type() : at::kBFloat16);
    ctx->saved_data["b"] = static_cast<int64_t>(bias.has_value() ? (codes.has_value() ? 5 : 3) : 0);
    return y;
  }
  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    check_backward();
    const variable_list v = ctx->get_saved_variables();
    const int64_t b = ctx->saved_data["b"].toInt();
    const bool need_x = ctx->needs_input_grad(0), need_b = b > 0 && ctx->needs_input_grad(b);
    Tensor dx, db;
    int8_backward(grads[0], Tensor(), Tensor(), v[0], v[1], ctx->saved_data["shape"].toIntVector(),
                  need_x ? &dx : nullptr, nullptr, at::kBFloat16, need_b ? &db : nullptr,
                  static_cast<at::ScalarType>(ctx->saved_data["bt"].toInt()));
    return {dx, Tensor(), Tensor(), Tensor(), Tensor(), db};
  }
};

void check_bias(const Tensor& b, int64_t N, const Tensor& x) {
  if (!b.defined()) return;
  TORCH_CHECK_TYPE(is_value(b.scalar_type()), "bias: expected bf16 or float32, got ", b.scalar_type());
  TORCH_CHECK_VALUE(b.dim() == 1 && b.size(0) == N, "bias: expected shape [", N, "], got ", b.sizes());
  TORCH_CHECK_VALUE(b.device() == x.device(), "bias: on ", b.device(), ", expected ", x.device());
}

// A backward pass has narrower limits than the forward: a call whose gradients are wanted
// is refused before its forward runs.
void check_int8_bwd(const Tensor& x, int64_t N) {
  const int64_t K = x.size(-1), M = x.numel() / K;
  TORCH_CHECK_VALUE(M == 0 || bitnet_int8_bwd_workspace_bytes(M, N, K) > 0, "int8_linear: ", M, " x ", K, " -> ", N,
                    " is too large for its backward pass, (rows + 256) * 2 * width <= 2^31 for each of its operands [",
                    M, ", ", K, "], [", N, ", ", K, "] and [", M, ", ", N,
                    "] with widths rounded up to 64: take fewer tokens at once, or torch.no_grad() for the forward alone");
}

Tensor int8_linear(const Tensor& x, const optional<Tensor>& codes, const optional<Tensor>& scales, const Tensor& weight,
                   const optional<Tensor>& bias) {
  const Tensor q = codes.value_or(Tensor()), s = scales.value_or(Tensor()), b = bias.value_or(Tensor());
  check_eager("int8_linear", {&x, &q, &s, &weight, &b});
  check_layer_input("int8_linear", x, q, s);
  TORCH_CHECK_TYPE(is_value(weight.scalar_type()), "weight: expected bf16 or float32, got ", weight.scalar_type());
  TORCH_CHECK_VALUE(weight.dim() == 2 && weight.size(1) == x.size(-1) && weight.size(0) >= 1,
                    "weight: expected [out_features, ", x.size(-1), "], got ", weight.sizes());
  TORCH_CHECK_VALUE(weight.device() == x.device(), "x and weight: must be GPU tensors of one device");
  check_bias(b, weight.size(0), x);
  if (wants_grad({&x, &weight, &b})) {
    check_int8_bwd(x, weight.size(0));
    return Int8Fn::apply(x, codes, scales, weight, bias);
  }
  const Rows r(x, q, s);
  const auto w = int8_weight(weight, &r);
  return int8_forward(r, x.sizes(), w.first, w.second, b);
}

Tensor int8_linear_inference(const Tensor& x, const optional<Tensor>& codes, const optional<Tensor>& scales,
                             const Tensor& w_q, const Tensor& s_w, int64_t in_features, const optional<Tensor>& bias) {
  const Tensor q = codes.value_or(Tensor()), s = scales.value_or(Tensor()), b = bias.value_or(Tensor());
  check_eager("int8_linear", {&x, &q, &s, &w_q, &s_w, &b});
  check_layer_input("int8_linear", x, q, s);
  TORCH_CHECK_VALUE(x.size(-1) == in_features, "x: expected a last dimension of ", in_features, ", got ", x.sizes());
  TORCH_CHECK_TYPE(w_q.scalar_type() == at::kChar && s_w.scalar_type() == at::kFloat,
                   "w_q: expected int8 and s_w float32, got ", w_q.scalar_type(), " and ", s_w.scalar_type());
  TORCH_CHECK_VALUE(w_q.dim() == 2 && w_q.size(0) >= 1 && w_q.size(1) == bitnet_k_pad(in_features) && s_w.dim() == 1 &&
                        s_w.size(0) == w_q.size(0),
                    "w_q: expected [out_features, ", bitnet_k_pad(in_features), "] and s_w [out_features], got ",
                    w_q.sizes(), " and ", s_w.sizes());
  TORCH_CHECK_VALUE(w_q.device() == x.device() && s_w.device() == x.device(),
                    "x, w_q and s_w: must be GPU tensors of one device");
  check_bias(b, w_q.size(0), x);
  const Tensor wq = aligned(w_q), sw = aligned(s_w);
  // a frozen module's bias wants a gradient in evaluation too: only that of x is looked at here
  if (wants_grad({&x})) check_int8_bwd(x, wq.size(0));
  if (wants_grad({&x, &b})) return Int8FrozenFn::apply(x, codes, scales, wq, sw, bias);
  const Rows r(x, q, s, true);
  if (r.M > 0) {
    On on(wq);
    r.quantize(on.stream);
  }
  return int8_forward(r, x.sizes(), wq, sw, b);
}

// The stored state of a weight, for the inference form.
std::pair<Tensor, Tensor> int8_quantize_weight(const Tensor& weight) {
  check_eager("int8_linear", {&weight});
  TORCH_CHECK_TYPE(is_value(weight.scalar_type()), "weight: expected bf16 or float32, got ", weight.scalar_type());
  TORCH_CHECK_VALUE(weight.dim() == 2 && weight.numel() > 0 && weight.is_cuda(),
                    "weight: expected a GPU tensor [out_features, in_features], got ", weight.sizes());
  at::NoGradGuard off;
  return int8_weight(weight, nullptr);
}

// --- the ternary layer of 8-bit rows ---------------------------------------------------------

struct Ternary {
  Tensor packed, gamma;
  explicit Ternary(const Tensor& weight) {
    const Tensor w = aligned(weight);
    const int64_t N = w.size(0), K = w.size(1);
    packed = at::empty({N, bitnet_k_pad(K) / 4}, w.options().dtype(at::kByte));
    gamma = at::empty({1}, w.options().dtype(at::kFloat));
    const size_t bytes = bitnet_ternarize_workspace_bytes(N, K);
    const Tensor ws = scratch(bytes, w);
    On on(w);
    check(bitnet_ternarize_pack(ptr(w), code(w.scalar_type()), N, K, static_cast<uint8_t*>(ptr(packed)), f32(gamma),
                                ptr(ws), bytes, on.stream));
  }
};

Tensor bitlinear_forward(const Rows& x, at::IntArrayRef shape, const Tensor& packed, const Tensor& gamma,
                         const Tensor& bias) {
  const int64_t N = packed.size(0);
  Tensor y = at::empty(with_last(shape, N), packed.options().dtype(at::kBFloat16));
  if (x.M == 0) return y;
  const Tensor b = bias.defined() ? aligned(bias.to(at::kBFloat16)) : Tensor();
  const size_t bytes = bitlinear_fwd_workspace_bytes(x.M, N, x.K);
  const Tensor ws = scratch(bytes, packed);
  On on(packed);
  check(bitlinear_fwd_bias(i8(x.q), f32(x.s), static_cast<uint8_t*>(ptr(packed)), f32(gamma), bf16(b), x.M, N, x.K,
                           bf16(y), nullptr, bytes ? ptr(ws) : nullptr, bytes, on.stream));
  return y;
}

void bitlinear_backward(const Tensor& grad, const Tensor& q, const Tensor& s, const Tensor& packed, const Tensor& gamma,
                        at::IntArrayRef shape, Tensor* dx, Tensor* dw, at::ScalarType wt, Tensor* db, at::ScalarType bt) {
  const int64_t N = packed.size(0), K = shape.back();
  const Tensor dY = aligned(rows(grad.to(at::kBFloat16)));
  const int64_t M = dY.size(0);
  const auto o = dY.options();
  if (dx) *dx = at::empty(shape, o);
  if (M == 0) {
    if (dw) *dw = at::zeros({N, K}, o.dtype(wt));
    if (db) *db = at::zeros({N}, o.dtype(bt));
    return;
  }
  if (dw) *dw = at::empty({N, K}, o.dtype(wt));
  if (db) *db = at::empty({N}, o.dtype(bt));
  On on(dY);
  if (dx || dw) {
    const size_t bytes = bitlinear_bwd_workspace_bytes(M, N, K);
    const Tensor ws = scratch(bytes, dY);
    check(bitlinear_bwd(bf16(dY), dw ? i8(q) : nullptr, dw ? f32(s) : nullptr, static_cast<uint8_t*>(ptr(packed)),
                        f32(gamma), M, N, K, dx ? bf16(*dx) : nullptr, dw ? ptr(*dw) : nullptr, code(wt),
                        bytes ? ptr(ws) : nullptr, bytes, on.stream));
  }
  if (db) check(bitlinear_bias_grad(bf16(dY), M, N, ptr(*db), code(bt), on.stream));
}

struct RowsBitLinearFn : torch::autograd::Function<RowsBitLinearFn> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const Tensor& codes, const Tensor& scales,
                        const Tensor& weight, const optional<Tensor>& bias) {
    const Rows r(x, codes, scales);
    const Ternary w(weight);
    Tensor y = bitlinear_forward(r, x.sizes(), w.packed, w.gamma, bias.value_or(Tensor()));
    ctx->save_for_backward({r.q, r.s, w.packed, w.gamma});
    ctx->saved_data["shape"] = x.sizes();
    ctx->saved_data["wt"] = static_cast<int64_t>(weight.scalar_type());
    ctx->saved_data["bt"] = static_cast<int64_t>(bias.has_value() ? bias->scalar_type() : at::kBFloat16);
    ctx->saved_data["b"] = bias.has_value();
    return y;
  }
  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    check_backward();
    const variable_list v = ctx->get_saved_variables();
    const bool need_x = ctx->needs_input_grad(0), need_w = ctx->needs_input_grad(3);
    const bool need_b = ctx->saved_data["b"].toBool() && ctx->needs_input_grad(4);
    Tensor dx, dw, db;
    bitlinear_backward(grads[0], v[0], v[1], v[2], v[3], ctx->saved_data["shape"].toIntVector(), need_x ? &dx : nullptr,
                       need_w ? &dw : nullptr, static_cast<at::ScalarType>(ctx->saved_data["wt"].toInt()),
                       need_b ? &db : nullptr, static_cast<at::ScalarType>(ctx->saved_data["bt"].toInt()));
    return {dx, Tensor(), Tensor(), dw, db};
  }
};

struct RowsFrozenBitLinearFn : torch::autograd::Function<RowsFrozenBitLinearFn> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const Tensor& codes, const Tensor& scales,
                        const Tensor& packed, const Tensor& gamma, const optional<Tensor>& bias) {
    Tensor y = bitlinear_forward(Rows(x, codes, scales), x.sizes(), packed, gamma, bias.value_or(Tensor()));
    ctx->save_for_backward({packed, gamma});
    ctx->saved_data["shape"] = x.sizes();
    ctx->saved_data["bt"] = static_cast<int64_t>(bias.has_value() ? bias->scalar_type() : at::kBFloat16);
    ctx->saved_data["b"] = bias.has_value();
    return y;
  }
  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    check_backward();
    const variable_list v = ctx->get_saved_variables();
    const bool need_b = ctx->saved_data["b"].toBool() && ctx->needs_input_grad(5);
    Tensor dx, db;
    bitlinear_backward(grads[0], Tensor(), Tensor(), v[0], v[1], ctx->saved_data["shape"].toIntVector(),
                       ctx->needs_input_grad(0) ? &dx : nullptr, nullptr, at::kBFloat16, need_b ? &db : nullptr,
                       static_cast<at::ScalarType>(ctx->saved_data["bt"].toInt()));
    return {dx, Tensor(), Tensor(), Tensor(), Tensor(), db};
  }
};

Tensor rows_bitlinear(const Tensor& x, const Tensor& codes, const Tensor& scales, const Tensor& weight,
                      const optional<Tensor>& bias) {
  const Tensor b = bias.value_or(Tensor());
  check_eager("BitLinear", {&x, &codes, &scales, &weight, &b});
  check_rows("BitLinear", x, codes, scales);
  TORCH_CHECK_TYPE(is_value(weight.scalar_type()), "weight: expected bf16 or float32, got ", weight.scalar_type());
  TORCH_CHECK_VALUE(weight.dim() == 2 && weight.size(1) == x.size(-1) && weight.size(0) >= 1,
                    "weight: expected [out_features, ", x.size(-1), "], got ", weight.sizes());
  TORCH_CHECK_VALUE(weight.device() == x.device(), "x and weight: must be GPU tensors of one device");
  check_bias(b, weight.size(0), x);
  if (wants_grad({&x, &weight, &b})) return RowsBitLinearFn::apply(x, codes, scales, weight, bias);
  const Ternary w(weight);
  return bitlinear_forward(Rows(x, codes, scales), x.sizes(), w.packed, w.gamma, b);
}

Tensor rows_bitlinear_inference(const Tensor& x, const Tensor& codes, const Tensor& scales, const Tensor& w_packed,
                                const Tensor& gamma_, int64_t in_features, const optional<Tensor>& bias) {
  const Tensor b = bias.value_or(Tensor());
  check_eager("BitLinear", {&x, &codes, &scales, &w_packed, &gamma_, &b});
  check_rows("BitLinear", x, codes, scales);
  TORCH_CHECK_VALUE(x.size(-1) == in_features, "x: expected a last dimension of ", in_features, ", got ", x.sizes());
  TORCH_CHECK_TYPE(w_packed.scalar_type() == at::kByte && gamma_.scalar_type() == at::kFloat,
                   "w_packed: expected uint8 and gamma float32, got ", w_packed.scalar_type(), " and ",
                   gamma_.scalar_type());
  TORCH_CHECK_VALUE(w_packed.dim() == 2 && w_packed.size(0) >= 1 &&
                        w_packed.size(1) == bitnet_k_pad(in_features) / 4 && gamma_.numel() == 1,
                    "w_packed: expected [out_features, ", bitnet_k_pad(in_features) / 4, "] and gamma [1], got ",
                    w_packed.sizes(), " and ", gamma_.sizes());
  TORCH_CHECK_VALUE(w_packed.device() == x.device() && gamma_.device() == x.device(),
                    "x, w_packed and gamma: must be GPU tensors of one device");
  check_bias(b, w_packed.size(0), x);
  const Tensor packed = aligned(w_packed), gamma = gamma_.contiguous();
  if (wants_grad({&x, &b})) return RowsFrozenBitLinearFn::apply(x, codes, scales, packed, gamma, bias);
  return bitlinear_forward(Rows(x, codes, scales), x.sizes(), packed, gamma, b);
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
  m.def("rows_values", &rows_values, free_gil);
  m.def("rms_norm", &rms_norm, free_gil);
  m.def("gated_bitlinear", &gated_bitlinear, free_gil);
  m.def("gated_bitlinear_inference", &gated_bitlinear_inference, free_gil);
  m.def("int8_linear", &int8_linear, free_gil);
  m.def("int8_linear_inference", &int8_linear_inference, free_gil);
  m.def("int8_quantize_weight", &int8_quantize_weight, free_gil);
  m.def("rows_bitlinear", &rows_bitlinear, free_gil);
  m.def("rows_bitlinear_inference", &rows_bitlinear_inference, free_gil);
}
