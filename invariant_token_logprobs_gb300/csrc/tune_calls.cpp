// tune_calls.cpp: the Python calls of tune.py on torch tensors, as train_calls.cpp is for
// train.py: argument checks, output allocation and the call into liblp's C ABI
// (include/lp_tune.h).  No step of a computation is here.
#include "calls.h"

#include "../../include/lp_tune.h"

namespace {

struct EntryPoints {
  decltype(&lp_layer_norm) layer_norm;
  decltype(&lp_layer_norm_backward_workspace_size) norm_workspace;
  decltype(&lp_layer_norm_backward) layer_norm_backward;
  decltype(&lp_preference_loss_workspace_size) preference_workspace;
  decltype(&lp_preference_loss) preference_loss;
  decltype(&lp_muon_workspace_size) muon_workspace;
  decltype(&lp_muon_step) muon_step;
} lp;

// The dtype of weight and bias, which is one.
int weights_of(const at::Tensor* weight, const at::Tensor* bias, int64_t d) {
  int dtype = LP_FLOAT32;
  if (weight != nullptr) {
    dtype = dtype_code(*weight, "weight");
    vector(weight, d, "weight", weight->scalar_type());
  }
  if (bias != nullptr) {
    dtype = dtype_code(*bias, "bias");
    vector(bias, d, "bias", bias->scalar_type());
    if (weight != nullptr && weight->scalar_type() != bias->scalar_type())
      type_error("weight and bias must have one dtype");
  }
  return dtype;
}

// residual, branch, weight, bias, eps, in_place
PyObject* layer_norm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    const at::Tensor& residual = required(v[0], "residual");
    const at::Tensor *branch = tensor(v[1], "branch"), *weight = tensor(v[2], "weight"),
                     *bias = tensor(v[3], "bias");
    const float eps = float(number(v[4]));
    const bool in_place = truth(v[5]);
    const at::Tensor& act = branch != nullptr ? *branch : residual;
    const c10::Device device = device_of(residual, {branch, weight, bias});
    const c10::cuda::CUDAGuard guard(device);
    if (residual.dim() != 2) value_error("expected a 2-D residual");
    const int64_t T = residual.size(0), d = residual.size(1);
    const int residual_dtype = dtype_code(residual, "residual"), act_dtype = dtype_code(act, "branch");
    const int weight_dtype = weights_of(weight, bias, d);
    const int64_t ld_residual = row_stride(&residual, T, d, "residual");
    const int64_t ld_branch = row_stride(branch, T, d, "branch");
    at::Tensor stream = residual, normed, mean, rstd;
    int64_t ld_stream = ld_residual;
    Tensors made(device);
    if (branch != nullptr && !in_place) {
      made.add(&stream, {T, d}, residual.scalar_type());
      ld_stream = d;
    }
    made.add(&normed, {T, d}, act.scalar_type());
    made.add(&mean, {T}, at::kFloat);
    made.add(&rstd, {T}, at::kFloat);
    made.allocate();
    check_status("lp_layer_norm",
                 lp.layer_norm(data(residual), ld_residual, residual_dtype, data(branch), ld_branch,
                               act_dtype, data(weight), data(bias), weight_dtype, T, d, eps,
                               branch != nullptr ? data(stream) : nullptr, ld_stream, data(normed),
                               d, floats(mean), floats(rstd), current_stream(device)));
    if (branch != nullptr && !in_place) return tuple_of({&normed, &stream, &mean, &rstd});
    if (branch != nullptr) written_in_place(&residual);
    PyObject* out = tuple_of({&normed, &normed, &mean, &rstd});  // the very object that was given
    PyObject* old = PyTuple_GET_ITEM(out, 1);
    Py_INCREF(v[0]);
    PyTuple_SET_ITEM(out, 1, v[0]);
    Py_DECREF(old);
    return out;
  });
}

// grad_normed, grad_residual, residual, mean, rstd, weight, bias, branch, weight_grads, workspace
PyObject* layer_norm_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const at::Tensor& grad_normed = required(v[0], "grad_normed");
    const at::Tensor* grad_residual = tensor(v[1], "grad_residual");
    const at::Tensor& residual = required(v[2], "residual");
    const at::Tensor &mean = required(v[3], "mean"), &rstd = required(v[4], "rstd");
    const at::Tensor *weight = tensor(v[5], "weight"), *bias = tensor(v[6], "bias");
    const bool branch = truth(v[7]), weight_grads = truth(v[8]);
    const at::Tensor* given = tensor(v[9], "workspace");
    const c10::Device device =
        device_of(residual, {&grad_normed, grad_residual, &mean, &rstd, weight, bias, given});
    const c10::cuda::CUDAGuard guard(device);
    if (residual.dim() != 2) value_error("expected a 2-D residual");
    const int64_t T = residual.size(0), d = residual.size(1);
    const int residual_dtype = dtype_code(residual, "residual");
    const int act_dtype = dtype_code(grad_normed, "grad_normed");
    const int weight_dtype = weights_of(weight, bias, d);
    if (!branch && act_dtype != residual_dtype)
      type_error("without a branch grad_normed has the residual's dtype");
    same_dtype(grad_residual, residual.scalar_type(), "grad_residual");
    vector(&mean, T, "mean");
    vector(&rstd, T, "rstd");
    const int64_t ld_residual = row_stride(&residual, T, d, "residual");
    const int64_t ld_normed = row_stride(&grad_normed, T, d, "grad_normed");
    const int64_t ld_grad = row_stride(grad_residual, T, d, "grad_residual");
    at::Tensor out, grad_branch, grad_weight, grad_bias, workspace;
    Tensors made(device);
    made.add(&out, {T, d}, residual.scalar_type());
    const bool cast = branch && act_dtype != residual_dtype;
    if (cast) made.add(&grad_branch, {T, d}, grad_normed.scalar_type());
    size_t bytes = 0;
    if (weight_grads && (weight != nullptr || bias != nullptr)) {
      if (weight != nullptr) made.add(&grad_weight, {d}, at::kFloat);
      if (bias != nullptr) made.add(&grad_bias, {d}, at::kFloat);
      if (given != nullptr) {
        workspace = *given;
        bytes = workspace_bytes(*given);
      } else {
        bytes = lp.norm_workspace(T, d);
        made.scratch(&workspace, bytes);
      }
    }
    made.allocate();
    const auto at = [](const at::Tensor& t) { return t.defined() ? data(t) : nullptr; };
    check_status("lp_layer_norm_backward",
                 lp.layer_norm_backward(
                     data(residual), ld_residual, residual_dtype, act_dtype, data(weight),
                     weight_dtype, T, d, floats(mean), floats(rstd), data(grad_normed), ld_normed,
                     data(grad_residual), ld_grad, data(out), d, at(grad_branch), d,
                     static_cast<float*>(at(grad_weight)), static_cast<float*>(at(grad_bias)),
                     at(workspace), bytes, current_stream(device)));
    return tuple_of({&out, branch && !cast ? &out : &grad_branch, &grad_weight, &grad_bias});
  });
}

// logp, cu_seqlens, ref_logp, mask, kind, average, halves, beta, margin, label_smoothing, nll_coef,
// workspace
PyObject* preference_loss(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    const at::Tensor& logp = required(v[0], "logp");
    const at::Tensor& cu_seqlens = required(v[1], "cu_seqlens");
    const at::Tensor *ref_logp = tensor(v[2], "ref_logp"), *mask = tensor(v[3], "mask"),
                     *given = tensor(v[11], "workspace");
    const int kind = int(integer(v[4]));
    const bool average = truth(v[5]), halves = truth(v[6]);
    const double beta = number(v[7]), margin = number(v[8]), smoothing = number(v[9]), nll = number(v[10]);
    if (logp.dim() != 1) value_error("expected a 1-D logp");
    const c10::Device device = device_of(logp, {&cu_seqlens, ref_logp, mask, given});
    const c10::cuda::CUDAGuard guard(device);
    const int64_t T = logp.size(0);
    vector(&logp, T, "logp");
    vector(ref_logp, T, "ref_logp");
    if (mask != nullptr)
      vector(mask, T, "mask", mask->scalar_type() == at::kByte ? at::kByte : at::kBool);
    if (cu_seqlens.dim() != 1 || cu_seqlens.size(0) < 1) value_error("cu_seqlens must be a vector of n + 1");
    const int64_t sequences = cu_seqlens.size(0) - 1;
    vector(&cu_seqlens, sequences + 1, "cu_seqlens", at::kLong);
    if (sequences % 2 != 0) value_error("the sequences must be pairs: an even number of them");
    at::Tensor stats, rewards, grad_logp, workspace;
    Tensors made(device);
    made.add(&stats, {6}, at::kFloat);
    made.add(&rewards, {sequences}, at::kFloat);
    made.add(&grad_logp, {T}, at::kFloat);
    size_t bytes;
    if (given != nullptr) {
      workspace = *given;
      bytes = workspace_bytes(*given);
    } else {
      bytes = lp.preference_workspace(T, sequences);
      made.scratch(&workspace, bytes);
    }
    made.allocate();
    check_status("lp_preference_loss",
                 lp.preference_loss(floats(logp), floats(ref_logp), static_cast<uint8_t*>(data(mask)),
                                    static_cast<int64_t*>(data(cu_seqlens)), T, sequences, kind, average,
                                    halves, beta, margin, smoothing, nll, floats(stats), floats(rewards),
                                    floats(grad_logp), data(workspace), bytes, current_stream(device)));
    return tuple_of({&stats, &rewards, &grad_logp});
  });
}

// The momenta that a plan's addresses point into: float32, each matrix's rounded up to whole lines of
// MUON_ALIGN elements.  `written` has the params, and bfloat16 copies.
void momenta_of(const at::Tensor& momenta, PyObject* written) {
  constexpr int64_t kAlign = 64;
  if (!PyTuple_Check(written)) type_error("expected a tuple of tensors");
  int64_t elements = 0;
  for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(written); ++i) {
    const at::Tensor& t = required(PyTuple_GET_ITEM(written, i), "a tensor of the step");
    if (t.scalar_type() == at::kFloat) elements += (t.numel() + kAlign - 1) / kAlign * kAlign;
  }
  vector(&momenta, elements, "momenta");
}

// plan_host, plan, momenta, lr, momentum, nesterov, steps, eps, written, grads, streams, captured
PyObject* muon_step(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    const at::Tensor &plan_host = required(v[0], "plan_host"), &plan = required(v[1], "plan"),
                     &momenta = required(v[2], "momenta");
    if (plan_host.is_cuda()) value_error("plan_host must be in host memory");
    const double lr = number(v[3]), momentum = number(v[4]), eps = number(v[7]);
    const bool nesterov = truth(v[5]);
    const int64_t steps = integer(v[6]);
    const c10::Device device = device_of(plan, {&momenta});
    momenta_of(momenta, v[8]);
    const c10::cuda::CUDAGuard guard(device);
    const c10::cuda::CUDAStream on = c10::cuda::getCurrentCUDAStream(device.index());
    keep_for_step(on, v[1], {&momenta}, v[8], v[9], v[10], v[11]);
    const size_t bytes = lp.muon_workspace(data(plan_host));
    const at::Tensor workspace = empty({std::max<int64_t>(int64_t(bytes), 256)}, at::kByte, device);
    check_status("lp_muon_step",
                 lp.muon_step(data(plan_host), data(plan), lr, momentum, nesterov,
                              int(std::max<int64_t>(std::min<int64_t>(steps, 1000), 0)), eps,
                              data(workspace), bytes, on.stream()));
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(v[8]); ++i)
      written_in_place(&required(PyTuple_GET_ITEM(v[8], i), "a tensor of the step"));
    written_in_place(&momenta);
    return THPVariable_Wrap(workspace);
  });
}

PyObject* bind(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return bind_table(reinterpret_cast<void**>(&lp), sizeof(lp) / sizeof(void*), v, n);
}
PyMethodDef methods[] = {method<bind>("bind"),
                         method<layer_norm>("layer_norm"),
                         method<layer_norm_backward>("layer_norm_backward"),
                         method<preference_loss>("preference_loss"),
                         method<muon_step>("muon_step"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tune_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__tune_calls(void) { return PyModule_Create(&module); }
