// experts_api.cu -- the C ABI (include/ccl.h) of a rank's own experts (sort,
// rows, products) and of the AdamW step: argument checks and parameter
// blocks.  Host code only; invalid arguments are rejected before any CUDA call.
#include <math.h>
#include <string.h>

#include "api_checks.h"
#include "device_common.cuh"

using namespace ccl;

namespace {

constexpr size_t kMaxWidth = size_t{1} << 28;  // elements of a row
using Spans = SpansOf<kMoeMaxRanks * 6>;

ccl_status_t check_rows(const size_t* tokens, int p, int k, size_t hidden, ccl_dtype_t dt) {
  EXPERTS_TRY(check_tokens(tokens, p, k));
  if (hidden == 0 || hidden > kMaxWidth) return report_error(CCL_ERR_INVALID_ARG, "hidden=%zu outside 1..2^28", hidden);
  return check_float_dtype(dt, "rows");
}

uint32_t capacity(size_t rows) { return static_cast<uint32_t>(std::min<size_t>(rows, 0x7FFFFFFFu)); }

}  // namespace

extern "C" ccl_status_t ccl_moe_sort(const int32_t* const* expert_ids, const size_t* tokens, int p, int k,
                                     int num_experts, const int32_t* first_expert, int32_t* const* offsets,
                                     int32_t* const* rows, void* stream) {
  CCL_TRACE();
  clear_last_error();
  EXPERTS_TRY(check_tokens(tokens, p, k));
  if (num_experts < 1 || num_experts > kSortMaxExperts)
    return report_error(CCL_ERR_INVALID_ARG, "num_experts=%d outside 1..%d", num_experts, kSortMaxExperts);
  if (offsets == nullptr) return bad("offsets is NULL");
  if (any_tokens(tokens, p) && (expert_ids == nullptr || rows == nullptr)) return bad("expert_ids or rows is NULL");
  MoeSortArgs a;
  Spans spans;
  memset(&a, 0, sizeof(a));
  for (int r = 0; r < p; ++r) {
    EXPERTS_TRY(check_buffer("offsets", r, offsets[r], 4));
    a.offsets[r] = offsets[r];
    a.first[r] = first_expert != nullptr ? first_expert[r] : 0;
    a.items[r] = static_cast<uint32_t>(tokens[r] * k);
    spans.add(offsets[r], (static_cast<uint64_t>(num_experts) + 1) * 4, true);
    if (tokens[r] == 0) continue;
    EXPERTS_TRY(check_buffer("expert_ids", r, expert_ids[r], 4));
    EXPERTS_TRY(check_buffer("rows", r, rows[r], 4));
    a.ids[r] = expert_ids[r];
    a.rows[r] = rows[r];
    spans.add(expert_ids[r], a.items[r] * 4ull, false);
    spans.add(rows[r], a.items[r] * 4ull, true);
  }
  if (spans.clash()) return bad("an output overlaps another buffer");
  a.p = p;
  a.num_experts = num_experts;
  return launched(launch_moe_sort(a, on(stream)), "MoE sort kernel");
}

extern "C" ccl_status_t ccl_moe_to_experts(const void* const* x, const int32_t* const* rows, const size_t* tokens,
                                           int p, int k, size_t hidden, ccl_dtype_t dt, void* const* sorted,
                                           const size_t* sorted_rows, void* stream) {
  CCL_TRACE();
  clear_last_error();
  EXPERTS_TRY(check_rows(tokens, p, k, hidden, dt));
  if (sorted_rows == nullptr) return bad("sorted_rows is NULL");
  if (!any_tokens(tokens, p)) return CCL_OK;
  if (x == nullptr || rows == nullptr || sorted == nullptr) return bad("x, rows or sorted is NULL");
  const size_t e = dt == CCL_F32 ? 4 : 2;
  MoeRowsArgs a;
  Spans spans;
  memset(&a, 0, sizeof(a));
  uintptr_t bits = hidden * e;
  for (int r = 0; r < p; ++r) {
    if (tokens[r] == 0 || sorted_rows[r] == 0) continue;
    EXPERTS_TRY(check_buffer("x", r, x[r], e));
    EXPERTS_TRY(check_buffer("rows", r, rows[r], 4));
    EXPERTS_TRY(check_buffer("sorted", r, sorted[r], e));
    a.x[r] = x[r];
    a.rows[r] = rows[r];
    a.out[r] = sorted[r];
    a.tokens[r] = static_cast<uint32_t>(tokens[r]);
    a.cap[r] = capacity(sorted_rows[r]);
    bits |= reinterpret_cast<uintptr_t>(x[r]) | reinterpret_cast<uintptr_t>(sorted[r]);
    spans.add(x[r], tokens[r] * hidden * e, false);
    spans.add(rows[r], tokens[r] * k * 4, false);
    spans.add(sorted[r], static_cast<uint64_t>(a.cap[r]) * hidden * e, true);
  }
  if (spans.clash()) return bad("sorted overlaps another buffer");
  a.hidden = hidden;
  a.p = p;
  a.k = k;
  return launched(launch_moe_to_experts(dt, on_grid(bits), a, on(stream)), "MoE to-experts kernel");
}

extern "C" ccl_status_t ccl_moe_from_experts(const void* const* y, const size_t* y_rows, const int32_t* const* rows,
                                             const float* const* weights, const size_t* tokens, int p, int k,
                                             size_t hidden, ccl_dtype_t dt, void* const* out, void* stream) {
  CCL_TRACE();
  clear_last_error();
  EXPERTS_TRY(check_rows(tokens, p, k, hidden, dt));
  if (y_rows == nullptr) return bad("y_rows is NULL");
  if (!any_tokens(tokens, p)) return CCL_OK;
  if (y == nullptr || rows == nullptr || out == nullptr) return bad("y, rows or out is NULL");
  const size_t e = dt == CCL_F32 ? 4 : 2;
  MoeRowsArgs a;
  Spans spans;
  memset(&a, 0, sizeof(a));
  uintptr_t bits = hidden * e;
  for (int r = 0; r < p; ++r) {
    if (tokens[r] == 0) continue;
    if (y_rows[r] != 0) {
      EXPERTS_TRY(check_buffer("y", r, y[r], e));
      a.y[r] = y[r];
    }
    EXPERTS_TRY(check_buffer("rows", r, rows[r], 4));
    EXPERTS_TRY(check_buffer("out", r, out[r], e));
    if (weights != nullptr) {
      EXPERTS_TRY(check_buffer("weights", r, weights[r], 4));
      a.weights[r] = weights[r];
      spans.add(weights[r], tokens[r] * k * 4, false);
    }
    a.rows[r] = rows[r];
    a.out[r] = out[r];
    a.tokens[r] = static_cast<uint32_t>(tokens[r]);
    a.cap[r] = capacity(y_rows[r]);
    bits |= reinterpret_cast<uintptr_t>(a.y[r]) | reinterpret_cast<uintptr_t>(out[r]);
    spans.add(a.y[r], static_cast<uint64_t>(a.cap[r]) * hidden * e, false);
    spans.add(rows[r], tokens[r] * k * 4, false);
    spans.add(out[r], tokens[r] * hidden * e, true);
  }
  if (spans.clash()) return bad("out overlaps another buffer");
  a.hidden = hidden;
  a.p = p;
  a.k = k;
  return launched(launch_moe_from_experts(dt, on_grid(bits), a, on(stream)), "MoE from-experts kernel");
}

extern "C" ccl_status_t ccl_moe_from_experts_grad(const void* const* dout, const void* const* y, const size_t* y_rows,
                                                  const int32_t* const* rows, const float* const* weights,
                                                  const size_t* tokens, int p, int k, size_t hidden, ccl_dtype_t dt,
                                                  void* const* dy, float* const* dweights, void* stream) {
  CCL_TRACE();
  clear_last_error();
  EXPERTS_TRY(check_rows(tokens, p, k, hidden, dt));
  if (y_rows == nullptr) return bad("y_rows is NULL");
  if ((dy == nullptr && dweights == nullptr) || !any_tokens(tokens, p)) return CCL_OK;
  if (dout == nullptr || rows == nullptr || (dweights != nullptr && y == nullptr)) return bad("dout, rows or y is NULL");
  const size_t e = dt == CCL_F32 ? 4 : 2;
  MoeRowsArgs a;
  Spans spans;
  memset(&a, 0, sizeof(a));
  uintptr_t bits = hidden * e;
  for (int r = 0; r < p; ++r) {
    if (tokens[r] == 0) continue;
    EXPERTS_TRY(check_buffer("dout", r, dout[r], e));
    EXPERTS_TRY(check_buffer("rows", r, rows[r], 4));
    a.x[r] = dout[r];
    a.rows[r] = rows[r];
    a.tokens[r] = static_cast<uint32_t>(tokens[r]);
    a.cap[r] = capacity(y_rows[r]);
    const uint64_t row_bytes = static_cast<uint64_t>(a.cap[r]) * hidden * e;
    if (y_rows[r] != 0 && dweights != nullptr) {
      EXPERTS_TRY(check_buffer("y", r, y[r], e));
      a.y[r] = y[r];
      spans.add(y[r], row_bytes, false);
    }
    if (y_rows[r] != 0 && dy != nullptr) {
      EXPERTS_TRY(check_buffer("dy", r, dy[r], e));
      a.out[r] = dy[r];
      spans.add(dy[r], row_bytes, true);
    }
    if (dweights != nullptr) {
      EXPERTS_TRY(check_buffer("dweights", r, dweights[r], 4));
      a.dweights[r] = dweights[r];
      spans.add(dweights[r], tokens[r] * k * 4, true);
    }
    if (weights != nullptr) {
      EXPERTS_TRY(check_buffer("weights", r, weights[r], 4));
      a.weights[r] = weights[r];
      spans.add(weights[r], tokens[r] * k * 4, false);
    }
    bits |= reinterpret_cast<uintptr_t>(dout[r]) | reinterpret_cast<uintptr_t>(a.y[r]) |
            reinterpret_cast<uintptr_t>(a.out[r]);
    spans.add(dout[r], tokens[r] * hidden * e, false);
    spans.add(rows[r], tokens[r] * k * 4, false);
  }
  if (spans.clash()) return bad("dy or dweights overlaps another buffer");
  a.hidden = hidden;
  a.p = p;
  a.k = k;
  return launched(launch_moe_from_experts_grad(dt, on_grid(bits), a, on(stream)), "MoE from-experts gradient kernel");
}

// ---------------------------------------------------------------- products
namespace {

ccl_status_t product(int kind, const void* const* first, const char* first_name, const void* const* second,
                     const char* second_name, const int32_t* const* offsets, const size_t* rows, int p,
                     int num_experts, size_t n, size_t contract, ccl_dtype_t out_dt, void* const* out,
                     const char* out_name, void* stream) {
  clear_last_error();
  if (p < 1 || p > kMoeMaxRanks) return report_error(CCL_ERR_INVALID_ARG, "p=%d outside 1..%d", p, kMoeMaxRanks);
  if (num_experts < 1 || num_experts > kSortMaxExperts)
    return report_error(CCL_ERR_INVALID_ARG, "num_experts=%d outside 1..%d", num_experts, kSortMaxExperts);
  constexpr size_t most = size_t{1} << 22;  // keeps every element count below 2^54
  if (n == 0 || n > most || contract == 0 || contract > most)
    return report_error(CCL_ERR_INVALID_ARG, "n=%zu or contract=%zu outside 1..2^22", n, contract);
  if (out_dt != CCL_F32 && out_dt != CCL_BF16)
    return out_dt == CCL_I32 ? report_error(CCL_ERR_UNSUPPORTED, "weight gradients are fp32 or bf16")
                             : report_error(CCL_ERR_INVALID_ARG, "unknown dtype %d", static_cast<int>(out_dt));
  if (rows == nullptr || offsets == nullptr) return bad("rows or offsets is NULL");
  const bool weights_out = kind == kProductGradWeight;
  bool any = weights_out;
  for (int r = 0; r < p; ++r) {
    if (rows[r] > 0x7FFFFF00ull) return report_error(CCL_ERR_INVALID_ARG, "rows[%d] must stay below 2^31 - 255", r);
    any = any || rows[r] != 0;
  }
  if (!any) return CCL_OK;
  if (first == nullptr || second == nullptr || out == nullptr)
    return report_error(CCL_ERR_INVALID_ARG, "%s, %s or %s is NULL", first_name, second_name, out_name);
  const uint64_t weight = static_cast<uint64_t>(num_experts) * n * contract;
  const size_t e = out_dt == CCL_F32 ? 4 : 2;
  ProductArgs a;
  Spans spans;
  memset(&a, 0, sizeof(a));
  for (int r = 0; r < p; ++r) {
    if (rows[r] == 0 && !weights_out) continue;
    EXPERTS_TRY(check_buffer("offsets", r, offsets[r], 4));
    EXPERTS_TRY(check_buffer(out_name, r, out[r], e));
    if (rows[r] != 0) {
      EXPERTS_TRY(check_buffer(first_name, r, first[r], 2));
      EXPERTS_TRY(check_buffer(second_name, r, second[r], 2));
    }
    a.b[r] = rows[r] != 0 ? first[r] : nullptr;
    a.a[r] = rows[r] != 0 ? second[r] : nullptr;
    a.out[r] = out[r];
    a.offsets[r] = offsets[r];
    a.rows[r] = static_cast<uint32_t>(rows[r]);
    const uint64_t in_cols = kind == kProductForward ? contract : n, out_cols = kind == kProductForward ? n : contract;
    spans.add(a.b[r], rows[r] * in_cols * 2, false);
    spans.add(a.a[r], weights_out ? rows[r] * contract * 2 : weight * 2, false);
    spans.add(offsets[r], (static_cast<uint64_t>(num_experts) + 1) * 4, false);
    spans.add(out[r], weights_out ? weight * e : rows[r] * out_cols * 2, true);
  }
  if (spans.clash()) return report_error(CCL_ERR_INVALID_ARG, "%s overlaps another buffer", out_name);
  a.n = n;
  a.contract = contract;
  a.p = p;
  a.num_experts = num_experts;
  return launched(launch_moe_product(kind, out_dt, a, on(stream)), "MoE product kernel");
}

}  // namespace

extern "C" ccl_status_t ccl_moe_product(const void* const* x, const int32_t* const* offsets, const void* const* w,
                                        const size_t* rows, int p, int num_experts, size_t n, size_t contract,
                                        void* const* y, void* stream) {
  CCL_TRACE();
  return product(kProductForward, x, "x", w, "w", offsets, rows, p, num_experts, n, contract, CCL_BF16, y, "y", stream);
}

extern "C" ccl_status_t ccl_moe_product_grad_input(const void* const* dy, const int32_t* const* offsets,
                                                   const void* const* w, const size_t* rows, int p, int num_experts,
                                                   size_t n, size_t contract, void* const* dx, void* stream) {
  CCL_TRACE();
  return product(kProductGradInput, dy, "dy", w, "w", offsets, rows, p, num_experts, n, contract, CCL_BF16, dx, "dx", stream);
}

extern "C" ccl_status_t ccl_moe_product_grad_weight(const void* const* dy, const void* const* x,
                                                    const int32_t* const* offsets, const size_t* rows, int p,
                                                    int num_experts, size_t n, size_t contract, ccl_dtype_t dw_dt,
                                                    void* const* dw, void* stream) {
  CCL_TRACE();
  return product(kProductGradWeight, dy, "dy", x, "x", offsets, rows, p, num_experts, n, contract, dw_dt, dw, "dw", stream);
}

// ------------------------------------------------------------------- AdamW
namespace {

ccl_status_t check_adamw_tensor(const ccl_adamw_tensor_t& t, size_t i, size_t pe, size_t ge, int bits) {
  const size_t se = bits == 8 ? 1 : 4;
  const uint64_t scales = bits == 8 ? (t.n + kAdamwBlock - 1) / kAdamwBlock * 4 : 0;
  struct {
    const char* name;
    const void* p;
    size_t align;
    uint64_t bytes;
  } b[] = {{"param", t.param, pe, t.n * pe},
           {"grad", t.grad, ge, t.n * ge},
           {"exp_avg", t.exp_avg, se, t.n * se},
           {"exp_avg_sq", t.exp_avg_sq, se, t.n * se},
           {"exp_avg_scale", t.exp_avg_scale, 4, scales},
           {"exp_avg_sq_scale", t.exp_avg_sq_scale, 4, scales},
           {"copy", t.copy, 2, t.copy != nullptr ? t.n * 2 : 0}};
  for (const auto& v : b) {
    if (v.bytes == 0) continue;
    if (v.p == nullptr) return report_error(CCL_ERR_INVALID_ARG, "tensor %zu: %s is NULL", i, v.name);
    if (reinterpret_cast<uintptr_t>(v.p) % v.align)
      return report_error(CCL_ERR_INVALID_ARG, "tensor %zu: %s is not %zu-byte aligned", i, v.name, v.align);
    for (const auto& w : b) {
      if (&w == &v) break;
      const uintptr_t x = reinterpret_cast<uintptr_t>(v.p), y = reinterpret_cast<uintptr_t>(w.p);
      if (w.bytes != 0 && x < y + w.bytes && y < x + v.bytes)
        return report_error(CCL_ERR_INVALID_ARG, "tensor %zu: %s overlaps %s", i, v.name, w.name);
    }
  }
  return CCL_OK;
}

// Launches over tensors[0..count): as many of them per launch as the block holds.
template <typename Args>
ccl_status_t adamw_launches(Args& a, const ccl_adamw_tensor_t* tensors, size_t count, int pdt, int gdt, int bits,
                            bool copy, void* stream) {
  size_t i = 0;
  while (i < count) {
    int m = 0;
    uint64_t chunks = 0;
    for (; i < count && m < Args::kCap; ++i) {
      const ccl_adamw_tensor_t& t = tensors[i];
      if (t.n == 0) continue;
      const uint64_t c = (t.n + kAdamwChunk - 1) / kAdamwChunk;
      if (chunks + c > 0x7FFFFFFFull) break;
      a.t[m] = {t.param, t.grad, t.exp_avg, t.exp_avg_sq, t.exp_avg_scale, t.exp_avg_sq_scale, t.copy, t.n};
      a.chunk0[m++] = static_cast<uint32_t>(chunks);
      chunks += c;
    }
    if (m == 0) break;
    a.chunk0[m] = static_cast<uint32_t>(chunks);
    a.count = m;
    EXPERTS_TRY(launched(launch_adamw(pdt, gdt, bits, copy, a, on(stream)), "AdamW kernel"));
  }
  return CCL_OK;
}

AdamwPair twice(double x) {
  const float f = static_cast<float>(x);
  uint32_t bits;
  memcpy(&bits, &f, sizeof(bits));
  return {static_cast<uint64_t>(bits) << 32 | bits};
}

template <typename Args>
ccl_status_t adamw_run(const ccl_adamw_tensor_t* tensors, size_t count, int pdt, int gdt, int bits, bool copy,
                       const ccl_adamw_hyper_t& h, void* stream) {
  Args a;  // entries past the launch's tensors are never read
  const double t = static_cast<double>(h.step);
  a.root_scale = static_cast<float>(1.0 / sqrt(1.0 - pow(h.beta2, t)));
  a.eps = static_cast<float>(h.eps);
  a.k = {twice(h.beta1), twice(1.0 - h.beta1), twice(h.beta2), twice(1.0 - h.beta2), twice(1.0 - h.lr * h.weight_decay),
         twice(-(h.lr / (1.0 - pow(h.beta1, t)))), twice(a.root_scale), twice(a.eps),
         twice(1.0), twice(-1.0), twice(0.5), twice(-0.5), twice(ldexp(1.0, -120))};
  a.dither = static_cast<uint32_t>(h.step * 2654435769ull);
  a.grad_scale = h.grad_scale;
  // with sqrt(v) 0 or in 2^-48 .. 2^20 the denominator stays in 2^-48 .. 2^30
  a.any_range = !(a.eps >= ldexpf(1.0f, -48) && a.eps <= ldexpf(1.0f, 28) && a.root_scale <= ldexpf(1.0f, 9));
  return adamw_launches(a, tensors, count, pdt, gdt, bits, copy, stream);
}

}  // namespace

extern "C" ccl_status_t ccl_adamw_step(const ccl_adamw_tensor_t* tensors, size_t count, ccl_dtype_t param_dt,
                                       ccl_dtype_t grad_dt, int state_bits, const ccl_adamw_hyper_t* hyper,
                                       void* stream) {
  CCL_TRACE();
  clear_last_error();
  if (hyper == nullptr) return bad("hyper is NULL");
  if ((param_dt != CCL_F32 && param_dt != CCL_BF16) || (grad_dt != CCL_F32 && grad_dt != CCL_BF16))
    return bad("parameters and gradients are fp32 or bf16");
  if (state_bits != 8 && state_bits != 32) return report_error(CCL_ERR_INVALID_ARG, "state_bits=%d is neither 8 nor 32", state_bits);
  const ccl_adamw_hyper_t& h = *hyper;
  if (!(isfinite(h.lr) && h.lr >= 0) || !(isfinite(h.eps) && h.eps >= 0) || !(isfinite(h.weight_decay) && h.weight_decay >= 0) ||
      !(h.beta1 >= 0 && h.beta1 < 1) || !(h.beta2 >= 0 && h.beta2 < 1))
    return bad("need lr, eps and weight_decay >= 0 and finite, beta1 and beta2 in [0, 1)");
  if (h.step == 0) return bad("step counts from 1");
  if (reinterpret_cast<uintptr_t>(h.grad_scale) & 3) return bad("grad_scale is not 4-byte aligned");
  if (count == 0) return CCL_OK;
  if (tensors == nullptr) return bad("tensors is NULL");
  const size_t pe = param_dt == CCL_F32 ? 4 : 2, ge = grad_dt == CCL_F32 ? 4 : 2;
  bool copy = false;
  for (size_t i = 0; i < count; ++i) {
    if (tensors[i].n >= (size_t{1} << 42)) return report_error(CCL_ERR_INVALID_ARG, "tensor %zu: n must stay below 2^42", i);
    copy = copy || tensors[i].copy != nullptr;
    EXPERTS_TRY(check_adamw_tensor(tensors[i], i, pe, ge, state_bits));
  }
  if (copy && param_dt != CCL_F32) return bad("a bf16 copy is written beside fp32 parameters only");
  return count <= static_cast<size_t>(AdamwSmall::kCap)
             ? adamw_run<AdamwSmall>(tensors, count, param_dt, grad_dt, state_bits, copy, h, stream)
             : adamw_run<AdamwLarge>(tensors, count, param_dt, grad_dt, state_bits, copy, h, stream);
}
