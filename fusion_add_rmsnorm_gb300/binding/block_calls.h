// Python wrappers of the block-scaled entry points (include/gbfuse_block.h).
#pragma once

#include "gbfuse_block.h"
#include "operands.h"

namespace {

constexpr int64_t kScaleBlock = 128;
int64_t blocks_of(int64_t n) { return (n + kScaleBlock - 1) / kScaleBlock; }

// The last dimension of a tensor, and how many such rows it holds.
struct Folded {
  int64_t rows, width;
};
Folded folded(const at::Tensor& t) {
  const int64_t w = t.dim() ? t.size(-1) : 0;
  return {w ? t.numel() / w : 0, w};
}

PyObject* add_rmsnorm_fp8_block(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&] {
    static const char* const names[12] = {"x",    "res_in", "res_out",   "q_out",     "scales", "mode",
                                          "weight", "gate", "ada_scale", "ada_shift", "eps",    "stream"};
    const Args<12> v("add_rmsnorm_fp8_block", names, 6, args, nargs, kwnames);
    const at::Tensor& x = tensor(v.at[0], names[0]);
    const int d = device_of(x);
    const auto [rows, hidden] = folded(x);
    auto bf16 = [&](int i, int64_t n) { return operand(v.at[i], n, at::kBFloat16, names[i], d); };
    const int64_t n = rows * hidden;
    void *xp = bf16(0, n), *in = bf16(1, n), *out = bf16(2, n);
    void* q = operand(v.at[3], n, at::kByte, names[3], d);
    void* s = operand(v.at[4], rows * blocks_of(hidden), at::kFloat, names[4], d);
    const int mode = narrow(v.at[5], names[5]);
    void *weight = bf16(6, hidden), *gate = bf16(7, hidden), *scale = bf16(8, hidden), *shift = bf16(9, hidden);
    const double eps = v.at[10] != Py_None ? real(v.at[10], names[10]) : 1e-6;
    void* st = stream(v.at[11], d);
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = gbfb_add_rmsnorm_fp8(xp, in, out, gate, mode, weight, scale, shift, static_cast<uint8_t*>(q),
                                  static_cast<float*>(s), rows, hidden, static_cast<float>(eps), st);
    Py_END_ALLOW_THREADS;
    return status;
  });
}

PyObject* gated_act_fp8_block(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&] {
    static const char* const names[5] = {"x", "q_out", "scales", "act", "stream"};
    const Args<5> v("gated_act_fp8_block", names, 3, args, nargs, kwnames);
    const at::Tensor &x = tensor(v.at[0], names[0]), &q = tensor(v.at[1], names[1]);
    const int d = device_of(x);
    const auto [rows, width] = folded(q);
    const int64_t given = folded(x).width;
    if (x.numel() && given != 2 * width)
      raise(PyExc_ValueError, "x: rows of %lld values, expected 2 * %lld", static_cast<long long>(given),
            static_cast<long long>(width));
    const void* xp = operand(v.at[0], 2 * rows * width, at::kBFloat16, names[0], d);
    void* qp = operand(v.at[1], rows * width, at::kByte, names[1], d);
    void* s = operand(v.at[2], rows * blocks_of(width), at::kFloat, names[2], d);
    const int act = v.at[3] != Py_None ? narrow(v.at[3], names[3]) : GBF_ACT_SILU;
    void* st = stream(v.at[4], d);
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = gbfb_gated_act_fp8(xp, static_cast<uint8_t*>(qp), static_cast<float*>(s), rows, width, act, st);
    Py_END_ALLOW_THREADS;
    return status;
  });
}

PyObject* quantize_fp8_block(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&] {
    static const char* const names[5] = {"x", "q_out", "scales", "block_rows", "stream"};
    const Args<5> v("quantize_fp8_block", names, 3, args, nargs, kwnames);
    const at::Tensor& x = tensor(v.at[0], names[0]);
    const int d = device_of(x);
    const auto [rows, width] = folded(x);
    const int per = v.at[3] != Py_None ? narrow(v.at[3], names[3]) : 1;
    const void* xp = operand(v.at[0], rows * width, at::kBFloat16, names[0], d);
    void* qp = operand(v.at[1], rows * width, at::kByte, names[1], d);
    // a block_rows that the call refuses has no extent to check
    const int64_t n = per > 0 ? (rows + per - 1) / per * blocks_of(width) : tensor(v.at[2], names[2]).numel();
    void* s = operand(v.at[2], n, at::kFloat, names[2], d);
    void* st = stream(v.at[4], d);
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = gbfb_quantize_fp8(xp, static_cast<uint8_t*>(qp), static_cast<float*>(s), rows, width, per, st);
    Py_END_ALLOW_THREADS;
    return status;
  });
}

PyObject* linear_fp8_block(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&] {
    static const char* const names[8] = {"xq", "x_scales", "wq", "w_scales", "bias", "y", "act", "stream"};
    const Args<8> v("linear_fp8_block", names, 6, args, nargs, kwnames);
    const at::Tensor &x = tensor(v.at[0], names[0]), &w = tensor(v.at[2], names[2]);
    const int d = device_of(x);
    const auto [m, k] = folded(x);
    if (w.dim() != 2 || w.size(1) != k) raise(PyExc_ValueError, "wq: expected [N, %lld]", static_cast<long long>(k));
    const int64_t n = w.size(0);
    const void* xp = operand(v.at[0], m * k, at::kByte, names[0], d);
    const void* xs = operand(v.at[1], m * blocks_of(k), at::kFloat, names[1], d);
    const void* wp = operand(v.at[2], n * k, at::kByte, names[2], d);
    const void* ws = operand(v.at[3], blocks_of(n) * blocks_of(k), at::kFloat, names[3], d);
    const void* bias = operand(v.at[4], n, at::kBFloat16, names[4], d);
    void* y = operand(v.at[5], m * n, at::kBFloat16, names[5], d);
    const int act = v.at[6] != Py_None ? narrow(v.at[6], names[6]) : GBF_ACT_GELU_TANH;
    void* st = stream(v.at[7], d);
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = gbfb_linear_fp8(static_cast<const uint8_t*>(xp), static_cast<const float*>(xs),
                             static_cast<const uint8_t*>(wp), static_cast<const float*>(ws), bias, y, m, n, k, act, st);
    Py_END_ALLOW_THREADS;
    return status;
  });
}

#define GBF_BLOCK_METHODS                                                                                              \
  {"add_rmsnorm_fp8_block", GBF_FAST(add_rmsnorm_fp8_block),                                                            \
   "add_rmsnorm_fp8_block(x, res_in, res_out, q_out, scales, mode, weight=None, gate=None, ada_scale=None, "           \
   "ada_shift=None, eps=1e-6, stream=None)\n--\n\n"                                                                    \
   "gbfb_add_rmsnorm_fp8 on [..., hidden] bf16 tensors (rows = every leading index);\n"                                \
   "q_out is uint8 E4M3 codes of the same shape, scales float32 [rows, ceil(hidden / 128)]."},                         \
  {"gated_act_fp8_block", GBF_FAST(gated_act_fp8_block),                                                               \
   "gated_act_fp8_block(x, q_out, scales, act=ACT_SILU, stream=None)\n--\n\n"                                          \
   "gbfb_gated_act_fp8: codes q_out[rows, d] and scales [rows, ceil(d / 128)] of\n"                                    \
   "act(x[:, :d]) * x[:, d:] for x [rows, 2d]."},                                                                      \
  {"quantize_fp8_block", GBF_FAST(quantize_fp8_block),                                                                 \
   "quantize_fp8_block(x, q_out, scales, block_rows=1, stream=None)\n--\n\n"                                           \
   "gbfb_quantize_fp8: codes q_out of x [..., d] and the scales of its blocks of\n"                                    \
   "block_rows (1, or 128 of a weight) x 128, [ceil(rows / block_rows), ceil(d / 128)]."},                             \
  {"linear_fp8_block", GBF_FAST(linear_fp8_block),                                                                     \
   "linear_fp8_block(xq, x_scales, wq, w_scales, bias, y, act=ACT_GELU_TANH, stream=None)\n--\n\n"                     \
   "gbfb_linear_fp8: y[..., N] = act(x @ w^T + bias) for uint8 codes xq [..., K] with\n"                               \
   "scales [rows, ceil(K / 128)] and wq [N, K] with [ceil(N / 128), ceil(K / 128)]."},

}  // namespace
