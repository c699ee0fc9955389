// train_calls.cpp: the Python calls of train.py on torch tensors.
//
// Argument checks, output allocation and the call into liblp's C ABI (include/lp_train.h),
// compiled because a call of the smallest operators takes 3 us on the GPU and its
// marshalling in Python took 16 to 30.  The entry points' addresses come from the loaded
// library (bind), so this file links no copy of it.  No step of a computation is here.
#include "calls.h"

namespace {

struct EntryPoints {
  decltype(&lp_residual_norm) residual_norm;
  decltype(&lp_residual_norm_backward_workspace_size) norm_workspace;
  decltype(&lp_residual_norm_backward) residual_norm_backward;
  decltype(&lp_policy_loss_workspace_size) policy_workspace;
  decltype(&lp_policy_loss) policy_loss;
  decltype(&lp_adamw_grad_norm_workspace_size) grad_norm_workspace;
  decltype(&lp_adamw_grad_norm) grad_norm;
  decltype(&lp_adamw_step) adamw_step;
  decltype(&lp_adamw_state_values) state_values;
} lp;

// What forward and backward of the residual norm share.
struct NormOperands {
  int64_t T, d;
  int residual_dtype, act_dtype, weight_dtype;
  int64_t ld_residual, ld_branch, ld_gate;
  NormOperands(const at::Tensor& residual, const at::Tensor* branch, const at::Tensor* gate,
               const at::Tensor* branch_weight, const at::Tensor* weight, const at::Tensor& act) {
    if (residual.dim() != 2) value_error("expected a 2-D residual");
    T = residual.size(0);
    d = residual.size(1);
    ld_gate = 0;
    if (gate != nullptr) {
      same_dtype(gate, act.scalar_type(), "gate");
      if (gate->dim() == 1) {
        vector(gate, d, "gate", act.scalar_type());
      } else {
        ld_gate = row_stride(gate, T, d, "gate");
        if (ld_gate < d) value_error("gate rows overlap: pass one row [d] for all");
      }
    }
    weight_dtype = LP_FLOAT32;
    if (weight != nullptr) {
      weight_dtype = dtype_code(*weight, "weight");
      vector(weight, d, "weight", weight->scalar_type());
    }
    if (branch_weight != nullptr) {
      weight_dtype = dtype_code(*branch_weight, "branch_weight");
      vector(branch_weight, d, "branch_weight", branch_weight->scalar_type());
      if (weight != nullptr && weight->scalar_type() != branch_weight->scalar_type())
        type_error("weight and branch_weight must have one dtype");
    }
    residual_dtype = dtype_code(residual, "residual");
    act_dtype = dtype_code(act, "activations");
    ld_residual = row_stride(&residual, T, d, "residual");
    ld_branch = row_stride(branch, T, d, "branch");
  }
};

// residual, branch, weight, branch_weight, gate, residual_scale, branch_scale, eps, in_place
PyObject* residual_norm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 9, [&] {
    const at::Tensor& residual = required(v[0], "residual");
    const at::Tensor *branch = tensor(v[1], "branch"), *weight = tensor(v[2], "weight"),
                     *branch_weight = tensor(v[3], "branch_weight"), *gate = tensor(v[4], "gate");
    const float a = float(number(v[5])), b = float(number(v[6])), eps = float(number(v[7]));
    const at::Tensor& act = branch != nullptr ? *branch : residual;
    const c10::Device device = device_of(residual, {branch, gate, branch_weight, weight});
    const c10::cuda::CUDAGuard guard(device);
    const NormOperands o(residual, branch, gate, branch_weight, weight, act);
    at::Tensor stream = residual, normed, rstd, branch_rstd;
    int64_t ld_stream = o.ld_residual;
    Tensors made(device);
    if (branch != nullptr && !truth(v[8])) {
      made.add(&stream, {o.T, o.d}, residual.scalar_type());
      ld_stream = o.d;
    }
    if (weight != nullptr) {
      made.add(&normed, {o.T, o.d}, act.scalar_type());
      made.add(&rstd, {o.T}, at::kFloat);
    }
    if (branch_weight != nullptr) made.add(&branch_rstd, {o.T}, at::kFloat);
    made.allocate();
    check_status("lp_residual_norm",
                 lp.residual_norm(data(residual), o.ld_residual, o.residual_dtype, data(branch),
                                  o.ld_branch, data(gate), o.ld_gate, o.act_dtype,
                                  data(branch_weight), data(weight), o.weight_dtype, o.T, o.d, a, b,
                                  eps, branch != nullptr ? data(stream) : nullptr, ld_stream,
                                  normed.defined() ? data(normed) : nullptr, o.d,
                                  branch_rstd.defined() ? floats(branch_rstd) : nullptr,
                                  rstd.defined() ? floats(rstd) : nullptr, current_stream(device)));
    if (branch != nullptr && truth(v[8])) written_in_place(&residual);
    if (branch == nullptr || truth(v[8])) {  // the very object that was given
      PyObject* out = tuple_of({&normed, &normed, &rstd, &branch_rstd});
      PyObject* old = PyTuple_GET_ITEM(out, 1);
      Py_INCREF(v[0]);
      PyTuple_SET_ITEM(out, 1, v[0]);
      Py_DECREF(old);
      return out;
    }
    return tuple_of({&normed, &stream, &rstd, &branch_rstd});
  });
}

// grad_normed, grad_residual, residual, rstd, branch, weight, branch_weight, branch_rstd, gate,
// residual_scale, branch_scale, weight_grads, workspace
PyObject* residual_norm_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    const at::Tensor *grad_normed = tensor(v[0], "grad_normed"),
                     *grad_residual = tensor(v[1], "grad_residual");
    const at::Tensor& residual = required(v[2], "residual");
    const at::Tensor *rstd = tensor(v[3], "rstd"), *branch = tensor(v[4], "branch"),
                     *weight = tensor(v[5], "weight"), *branch_weight = tensor(v[6], "branch_weight"),
                     *branch_rstd = tensor(v[7], "branch_rstd"), *gate = tensor(v[8], "gate");
    const float a = float(number(v[9])), b = float(number(v[10]));
    const bool weight_grads = truth(v[11]);
    const at::Tensor* given = tensor(v[12], "workspace");
    const at::Tensor& act = branch != nullptr ? *branch : residual;
    const c10::Device device = device_of(residual, {grad_normed, grad_residual, branch, gate, weight,
                                                    branch_weight, rstd, branch_rstd, given});
    const c10::cuda::CUDAGuard guard(device);
    const NormOperands o(residual, branch, gate, branch_weight, weight, act);
    same_dtype(grad_normed, act.scalar_type(), "grad_normed");
    same_dtype(grad_residual, residual.scalar_type(), "grad_residual");
    vector(rstd, o.T, "rstd");
    vector(branch_rstd, o.T, "branch_rstd");
    const int64_t ld_normed = row_stride(grad_normed, o.T, o.d, "grad_normed");
    const int64_t ld_grad = row_stride(grad_residual, o.T, o.d, "grad_residual");
    at::Tensor out, grad_branch, grad_gate, grad_weight, grad_branch_weight, workspace;
    Tensors made(device);
    made.add(&out, {o.T, o.d}, residual.scalar_type());
    if (branch != nullptr) made.add(&grad_branch, {o.T, o.d}, act.scalar_type());
    if (gate != nullptr && o.ld_gate != 0) made.add(&grad_gate, {o.T, o.d}, gate->scalar_type());
    size_t bytes = 0;
    if (weight_grads) {
      if (gate != nullptr && o.ld_gate == 0) made.add(&grad_gate, {o.d}, at::kFloat);
      if (weight != nullptr) made.add(&grad_weight, {o.d}, at::kFloat);
      if (branch_weight != nullptr) made.add(&grad_branch_weight, {o.d}, at::kFloat);
      if (given != nullptr) {
        workspace = *given;
        bytes = workspace_bytes(*given);
      } else {
        bytes = lp.norm_workspace(o.T, o.d);
        made.scratch(&workspace, bytes);
      }
    }
    made.allocate();
    const auto at = [](const at::Tensor& t) { return t.defined() ? data(t) : nullptr; };
    check_status(
        "lp_residual_norm_backward",
        lp.residual_norm_backward(
            weight != nullptr ? data(residual) : nullptr, o.ld_residual, o.residual_dtype,
            data(branch), o.ld_branch, data(gate), o.ld_gate, o.act_dtype, data(branch_weight),
            data(weight), o.weight_dtype, o.T, o.d, a, b, floats(branch_rstd), floats(rstd),
            data(grad_normed), ld_normed, data(grad_residual), ld_grad, data(out), o.d,
            at(grad_branch), o.d, at(grad_gate), o.d, static_cast<float*>(at(grad_branch_weight)),
            static_cast<float*>(at(grad_weight)), at(workspace), bytes, current_stream(device)));
    return tuple_of({&out, &grad_branch, &grad_weight, &grad_branch_weight, &grad_gate});
  });
}

// logp, old_logp, advantages, mask, ref_logp, entropy, cu_seqlens, by_sequence, per_sequence,
// clip_low, clip_high, kl_coef, entropy_coef, workspace
PyObject* policy_loss(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 14, [&] {
    const at::Tensor& logp = required(v[0], "logp");
    const at::Tensor& old_logp = required(v[1], "old_logp");
    const at::Tensor& advantages = required(v[2], "advantages");
    const at::Tensor *mask = tensor(v[3], "mask"), *ref_logp = tensor(v[4], "ref_logp"),
                     *entropy = tensor(v[5], "entropy"), *cu_seqlens = tensor(v[6], "cu_seqlens"),
                     *given = tensor(v[13], "workspace");
    const bool by_sequence = truth(v[7]), per_sequence = truth(v[8]);
    const double low = number(v[9]), high = number(v[10]), kl = number(v[11]), ent = number(v[12]);
    if (logp.dim() != 1) value_error("expected a 1-D logp");
    const c10::Device device =
        device_of(logp, {&old_logp, &advantages, mask, ref_logp, entropy, cu_seqlens, given});
    const c10::cuda::CUDAGuard guard(device);
    const int64_t T = logp.size(0);
    vector(&logp, T, "logp");
    vector(&old_logp, T, "old_logp");
    vector(ref_logp, T, "ref_logp");
    vector(entropy, T, "entropy");
    int64_t sequences = 0;
    if (by_sequence || per_sequence) {
      if (cu_seqlens == nullptr || cu_seqlens->dim() != 1 || cu_seqlens->size(0) < 1)
        value_error("cu_seqlens [n + 1] is needed");
      sequences = cu_seqlens->size(0) - 1;
      vector(cu_seqlens, sequences + 1, "cu_seqlens", at::kLong);
    } else {
      cu_seqlens = nullptr;
    }
    vector(&advantages, per_sequence ? sequences : T, "advantages");
    if (mask != nullptr)
      vector(mask, T, "mask", mask->scalar_type() == at::kByte ? at::kByte : at::kBool);
    at::Tensor stats, grad_logp, grad_entropy, workspace;
    Tensors made(device);
    made.add(&stats, {5}, at::kFloat);
    made.add(&grad_logp, {T}, at::kFloat);
    if (entropy != nullptr) made.add(&grad_entropy, {T}, at::kFloat);
    size_t bytes;
    if (given != nullptr) {
      workspace = *given;
      bytes = workspace_bytes(*given);
    } else {
      bytes = lp.policy_workspace(T, sequences);
      made.scratch(&workspace, bytes);
    }
    made.allocate();
    check_status("lp_policy_loss",
                 lp.policy_loss(floats(logp), floats(old_logp), floats(ref_logp), floats(entropy),
                                floats(advantages), per_sequence, static_cast<uint8_t*>(data(mask)),
                                static_cast<int64_t*>(data(cu_seqlens)), T, sequences,
                                by_sequence ? LP_REDUCE_SEQUENCE : LP_REDUCE_TOKEN, low, high, kl, ent,
                                floats(stats), floats(grad_logp),
                                grad_entropy.defined() ? floats(grad_entropy) : nullptr,
                                data(workspace), bytes, current_stream(device)));
    return tuple_of({&stats, &grad_logp, &grad_entropy});
  });
}

// plan, n_tensors, state_elements, state_bits, exp_avg, exp_avg_sq, exp_avg_scale,
// exp_avg_sq_scale, lr, beta1, beta2, eps, step, seed, max_norm or None, written, grads, streams,
// captured: the norm's tensor or None
PyObject* adamw_step(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 19, [&] {
    const at::Tensor& plan = required(v[0], "plan");
    const int64_t tensors = integer(v[1]), elements = integer(v[2]);
    const at::Tensor &m = required(v[4], "exp_avg"), &u = required(v[5], "exp_avg_sq");
    const at::Tensor *m_scale = tensor(v[6], "exp_avg_scale"), *u_scale = tensor(v[7], "exp_avg_sq_scale");
    const uint64_t seed = PyLong_AsUnsignedLongLong(v[13]);
    if (PyErr_Occurred()) throw Refused{};
    const c10::Device device = device_of(plan, {&m, &u, m_scale, u_scale});
    const c10::cuda::CUDAGuard guard(device);
    const c10::cuda::CUDAStream on = c10::cuda::getCurrentCUDAStream(device.index());
    void* stream = on.stream();
    keep_for_step(on, v[0], {&m, &u, m_scale, u_scale}, v[15], v[16], v[17], v[18]);
    at::Tensor norm;
    const float* scale = nullptr;
    if (v[14] != Py_None) {
      const size_t bytes = lp.grad_norm_workspace(elements);
      at::Tensor workspace;
      Tensors made(device);
      made.add(&norm, {2}, at::kFloat);
      made.scratch(&workspace, bytes);
      made.allocate();
      check_status("lp_adamw_grad_norm",
                   lp.grad_norm(data(plan), tensors, elements, float(number(v[14])), floats(norm),
                                data(workspace), bytes, stream));
      scale = floats(norm) + 1;
      norm = norm.select(0, 0);
    }
    check_status("lp_adamw_step",
                 lp.adamw_step(data(plan), tensors, elements, int(integer(v[3])), data(m), data(u),
                               floats(m_scale), floats(u_scale), number(v[8]), number(v[9]),
                               number(v[10]), number(v[11]), integer(v[12]), seed, scale, stream));
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(v[15]); ++i)
      written_in_place(&required(PyTuple_GET_ITEM(v[15], i), "a tensor of the step"));
    for (const at::Tensor* t : {&m, &u, m_scale, u_scale}) written_in_place(t);
    if (!norm.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(norm);
  });
}

// exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale of 8 bits: their values
PyObject* adamw_state_values(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 4, [&] {
    const at::Tensor &m = required(v[0], "exp_avg"), &u = required(v[1], "exp_avg_sq"),
                     &m_scale = required(v[2], "exp_avg_scale"),
                     &u_scale = required(v[3], "exp_avg_sq_scale");
    const c10::Device device = device_of(m, {&u, &m_scale, &u_scale});
    const c10::cuda::CUDAGuard guard(device);
    const int64_t elements = m.numel();
    at::Tensor values, squares;
    Tensors made(device);
    made.add(&values, {elements}, at::kFloat);
    made.add(&squares, {elements}, at::kFloat);
    made.allocate();
    for (const at::Tensor* t : {&m, &u, &m_scale, &u_scale})
      used_on(c10::cuda::getCurrentCUDAStream(device.index()), t);
    check_status("lp_adamw_state_values",
                 lp.state_values(data(m), data(u), floats(m_scale), floats(u_scale), elements,
                                 floats(values), floats(squares), current_stream(device)));
    return tuple_of({&values, &squares});
  });
}

PyObject* bind(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return bind_table(reinterpret_cast<void**>(&lp), sizeof(lp) / sizeof(void*), v, n);
}
PyMethodDef methods[] = {method<bind>("bind"),
                         method<residual_norm>("residual_norm"),
                         method<residual_norm_backward>("residual_norm_backward"),
                         method<policy_loss>("policy_loss"),
                         method<adamw_step>("adamw_step"),
                         method<adamw_state_values>("adamw_state_values"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_train_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__train_calls(void) { return PyModule_Create(&module); }
