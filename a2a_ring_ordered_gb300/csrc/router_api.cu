// router_api.cu -- the C ABI (include/ccl.h) of what stands before the
// experts: the router's choice with its balance loss, and the layer norm.
// Argument checks and parameter blocks; host code only, invalid arguments are
// rejected before any CUDA call.
#include <math.h>
#include <string.h>

#include "api_checks.h"

using namespace ccl;

namespace ccl {

void cut_rows(RankParts* parts, const size_t* rows, int p, uint32_t most, uint32_t least, bool all) {
  uint64_t total = 0;
  for (int r = 0; r < p; ++r) total += rows[r];
  uint32_t at = 0;
  for (int r = 0; r < p; ++r) {
    parts->first[r] = at;
    parts->rows[r] = static_cast<uint32_t>(rows[r]);
    if (rows[r] != 0) {
      // rows < 2^31 and most < 2^16: the product fits
      const uint64_t share = rows[r] * most / total, wanted = (rows[r] + least - 1) / least;
      at += static_cast<uint32_t>(std::max<uint64_t>(1, std::min(share, wanted)));
    } else if (all) {
      ++at;
    }
  }
  parts->first[p] = at;
}

}  // namespace ccl

namespace {

void take_rows(RankParts* parts, const size_t* rows, int p) {
  for (int r = 0; r < p; ++r) parts->rows[r] = static_cast<uint32_t>(rows[r]);
}

// ------------------------------------------------------------------ router
using GateSpans = SpansOf<kMoeMaxRanks * 7 + 1>;

ccl_status_t check_router(const size_t* tokens, int p, int k, int num_experts, ccl_dtype_t dt, ccl_score_t score) {
  EXPERTS_TRY(check_tokens(tokens, p, k));
  if (num_experts < 1 || num_experts > kSortMaxExperts)
    return report_error(CCL_ERR_INVALID_ARG, "num_experts=%d outside 1..%d", num_experts, kSortMaxExperts);
  if (k > num_experts) return report_error(CCL_ERR_INVALID_ARG, "k=%d of %d experts", k, num_experts);
  if (score != CCL_SCORE_SOFTMAX && score != CCL_SCORE_SIGMOID)
    return report_error(CCL_ERR_INVALID_ARG, "unknown score %d", static_cast<int>(score));
  return check_float_dtype(dt, "logits");
}

// Whether logits[r] are there, and their place in the block and the spans.
ccl_status_t take_logits(GateArgs* a, GateSpans* spans, uintptr_t* bits, const void* const* logits, int r, size_t tokens,
                         int num_experts, size_t e) {
  if (logits == nullptr) return bad("logits is NULL");
  EXPERTS_TRY(check_buffer("logits", r, logits[r], e));
  a->logits[r] = logits[r];
  *bits |= reinterpret_cast<uintptr_t>(logits[r]);
  spans->add(logits[r], tokens * num_experts * e, false);
  return CCL_OK;
}

// The loss's outputs and workspace.
ccl_status_t take_balance(BalanceJoinArgs* j, GateSpans* spans, int p, int k, int num_experts, const size_t* tokens,
                          int together, int32_t* const* counts, float* const* losses, const void* workspace,
                          size_t workspace_bytes) {
  if (counts == nullptr || losses == nullptr) return bad("counts and losses are given together");
  uint64_t pairs = 0;
  for (int r = 0; r < p; ++r) {
    EXPERTS_TRY(check_buffer("counts", r, counts[r], 4));
    EXPERTS_TRY(check_buffer("losses", r, losses[r], 4));
    j->counts[r] = counts[r];
    j->losses[r] = losses[r];
    spans->add(counts[r], (static_cast<uint64_t>(num_experts) + 1) * 4, true);
    spans->add(losses[r], 4, true);
    pairs += tokens[r] * k;
  }
  if (together && pairs > 0x7FFFFFFFull) return bad("the ranks' tokens * k together must stay below 2^31");
  const size_t need = ccl_moe_balance_workspace_bytes(p, num_experts);
  if (workspace == nullptr || workspace_bytes < need)
    return report_error(CCL_ERR_INVALID_ARG, "workspace of %zu bytes needed", need);
  if (reinterpret_cast<uintptr_t>(workspace) & 15) return bad("workspace is not 16-byte aligned");
  spans->add(workspace, need, true);
  j->p = p;
  j->k = k;
  j->num_experts = num_experts;
  j->together = together != 0;
  return CCL_OK;
}

ccl_status_t run_balance(const GateArgs& a, BalanceJoinArgs* j, void* stream) {
  memcpy(j->first, a.parts.first, sizeof(j->first));
  j->partial = a.partial;
  return launched(launch_balance_join(*j, on(stream)), "balance join kernel");
}

}  // namespace

extern "C" size_t ccl_moe_balance_workspace_bytes(int p, int num_experts) {
  if (p < 1 || p > kMoeMaxRanks || num_experts < 1 || num_experts > kSortMaxExperts) return 0;
  return (kBalanceParts + static_cast<size_t>(p)) * balance_part_words(num_experts) * 4;
}

extern "C" ccl_status_t ccl_moe_gate(const void* const* logits, const size_t* tokens, int p, int k, int num_experts,
                                     ccl_dtype_t dt, ccl_score_t score, int normalize, float scale,
                                     int32_t* const* ids, float* const* gates, int together, int32_t* const* counts,
                                     float* const* losses, void* workspace, size_t workspace_bytes, void* stream) {
  CCL_TRACE();
  clear_last_error();
  EXPERTS_TRY(check_router(tokens, p, k, num_experts, dt, score));
  if (!isfinite(scale)) return bad("scale must be finite");
  const bool balance = counts != nullptr || losses != nullptr;
  if (!balance && !any_tokens(tokens, p)) return CCL_OK;
  if (any_tokens(tokens, p) && (ids == nullptr || gates == nullptr)) return bad("ids or gates is NULL");
  const size_t e = dt == CCL_F32 ? 4 : 2;
  GateArgs a;
  BalanceJoinArgs j;
  GateSpans spans;
  memset(&a, 0, sizeof(a));
  memset(&j, 0, sizeof(j));
  uintptr_t bits = num_experts * e;
  for (int r = 0; r < p; ++r) {
    if (tokens[r] == 0) continue;
    EXPERTS_TRY(take_logits(&a, &spans, &bits, logits, r, tokens[r], num_experts, e));
    EXPERTS_TRY(check_buffer("ids", r, ids[r], 4));
    EXPERTS_TRY(check_buffer("gates", r, gates[r], 4));
    a.ids[r] = ids[r];
    a.gates[r] = gates[r];
    spans.add(ids[r], tokens[r] * k * 4, true);
    spans.add(gates[r], tokens[r] * k * 4, true);
  }
  if (balance)
    EXPERTS_TRY(take_balance(&j, &spans, p, k, num_experts, tokens, together, counts, losses, workspace, workspace_bytes));
  if (spans.clash()) return bad("an output overlaps another buffer");
  a.partial = static_cast<float*>(workspace);
  a.scale = scale;
  a.p = p;
  a.k = k;
  a.num_experts = num_experts;
  a.score = score;
  a.normalize = normalize != 0;
  take_rows(&a.parts, tokens, p);
  a.vec = on_grid(bits);
  EXPERTS_TRY(launched(launch_gate(dt, true, balance, &a, on(stream)), "MoE gate kernel"));
  return balance ? run_balance(a, &j, stream) : CCL_OK;
}

extern "C" ccl_status_t ccl_moe_balance(const void* const* logits, const int32_t* const* ids, const size_t* tokens,
                                        int p, int k, int num_experts, ccl_dtype_t dt, ccl_score_t score, int together,
                                        int32_t* const* counts, float* const* losses, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  CCL_TRACE();
  clear_last_error();
  EXPERTS_TRY(check_router(tokens, p, k, num_experts, dt, score));
  if (any_tokens(tokens, p) && ids == nullptr) return bad("ids is NULL");
  const size_t e = dt == CCL_F32 ? 4 : 2;
  GateArgs a;
  BalanceJoinArgs j;
  GateSpans spans;
  memset(&a, 0, sizeof(a));
  memset(&j, 0, sizeof(j));
  uintptr_t bits = num_experts * e;
  for (int r = 0; r < p; ++r) {
    if (tokens[r] == 0) continue;
    EXPERTS_TRY(take_logits(&a, &spans, &bits, logits, r, tokens[r], num_experts, e));
    EXPERTS_TRY(check_buffer("ids", r, ids[r], 4));
    a.ids_in[r] = ids[r];
    spans.add(ids[r], tokens[r] * k * 4, false);
  }
  EXPERTS_TRY(take_balance(&j, &spans, p, k, num_experts, tokens, together, counts, losses, workspace, workspace_bytes));
  if (spans.clash()) return bad("an output overlaps another buffer");
  a.partial = static_cast<float*>(workspace);
  a.p = p;
  a.k = k;
  a.num_experts = num_experts;
  a.score = score;
  take_rows(&a.parts, tokens, p);
  a.vec = on_grid(bits);
  EXPERTS_TRY(launched(launch_gate(dt, false, true, &a, on(stream)), "MoE balance kernel"));
  return run_balance(a, &j, stream);
}

namespace {

ccl_status_t router_grad(const void* const* logits, const int32_t* const* ids, const float* const* dgates,
                         const size_t* tokens, int p, int k, int num_experts, ccl_dtype_t dt, ccl_score_t score,
                         int normalize, float scale, const int32_t* const* counts, const float* const* dlosses,
                         float balance_scale, void* const* dlogits, bool gates, const char* what, void* stream) {
  clear_last_error();
  EXPERTS_TRY(check_router(tokens, p, k, num_experts, dt, score));
  if (!isfinite(scale) || !isfinite(balance_scale)) return bad("scales must be finite");
  const bool balance = counts != nullptr;
  if (!balance && !gates) return bad("counts is NULL");
  if (!balance && dlosses != nullptr) return bad("dlosses needs counts");
  if (!any_tokens(tokens, p)) return CCL_OK;
  if (dlogits == nullptr || (gates && (ids == nullptr || dgates == nullptr))) return bad("ids, dgates or dlogits is NULL");
  const size_t e = dt == CCL_F32 ? 4 : 2;
  GateArgs a;
  GateSpans spans;
  memset(&a, 0, sizeof(a));
  uintptr_t bits = num_experts * e;
  for (int r = 0; r < p; ++r) {
    if (tokens[r] == 0) continue;
    EXPERTS_TRY(take_logits(&a, &spans, &bits, logits, r, tokens[r], num_experts, e));
    EXPERTS_TRY(check_buffer("dlogits", r, dlogits[r], e));
    a.dlogits[r] = dlogits[r];
    bits |= reinterpret_cast<uintptr_t>(dlogits[r]);
    spans.add(dlogits[r], tokens[r] * num_experts * e, true);
    if (gates) {
      EXPERTS_TRY(check_buffer("ids", r, ids[r], 4));
      EXPERTS_TRY(check_buffer("dgates", r, dgates[r], 4));
      a.ids_in[r] = ids[r];
      a.dgates[r] = dgates[r];
      spans.add(ids[r], tokens[r] * k * 4, false);
      spans.add(dgates[r], tokens[r] * k * 4, false);
    }
    if (balance) {
      EXPERTS_TRY(check_buffer("counts", r, counts[r], 4));
      a.counts[r] = counts[r];
      spans.add(counts[r], (static_cast<uint64_t>(num_experts) + 1) * 4, false);
      if (dlosses != nullptr) {
        EXPERTS_TRY(check_buffer("dlosses", r, dlosses[r], 4));
        a.dlosses[r] = dlosses[r];
        spans.add(dlosses[r], 4, false);
      }
    }
  }
  if (spans.clash()) return bad("dlogits overlaps another buffer");
  a.scale = scale;
  a.balance_scale = balance_scale;
  a.p = p;
  a.k = k;
  a.num_experts = num_experts;
  a.score = score;
  a.normalize = normalize != 0;
  take_rows(&a.parts, tokens, p);
  a.vec = on_grid(bits);
  return launched(launch_gate_grad(dt, gates, balance, &a, on(stream)), what);
}

}  // namespace

extern "C" ccl_status_t ccl_moe_gate_grad(const void* const* logits, const int32_t* const* ids,
                                          const float* const* dgates, const size_t* tokens, int p, int k,
                                          int num_experts, ccl_dtype_t dt, ccl_score_t score, int normalize,
                                          float scale, const int32_t* const* counts, const float* const* dlosses,
                                          float balance_scale, void* const* dlogits, void* stream) {
  CCL_TRACE();
  return router_grad(logits, ids, dgates, tokens, p, k, num_experts, dt, score, normalize, scale, counts, dlosses,
                     balance_scale, dlogits, true, "MoE gate gradient kernel", stream);
}

extern "C" ccl_status_t ccl_moe_balance_grad(const void* const* logits, const int32_t* const* counts,
                                             const float* const* dlosses, const size_t* tokens, int p, int k,
                                             int num_experts, ccl_dtype_t dt, ccl_score_t score, float scale,
                                             void* const* dlogits, void* stream) {
  CCL_TRACE();
  return router_grad(logits, nullptr, nullptr, tokens, p, k, num_experts, dt, score, 0, 1.0f, counts, dlosses, scale,
                     dlogits, false, "MoE balance gradient kernel", stream);
}

// -------------------------------------------------------------- layer norm
namespace {

using NormSpans = SpansOf<kMoeMaxRanks * 9 + 1>;

ccl_status_t check_norm(const size_t* rows, int p, size_t cols, ccl_dtype_t dt, ccl_dtype_t weight_dt) {
  if (p < 1 || p > kMoeMaxRanks) return report_error(CCL_ERR_INVALID_ARG, "p=%d outside 1..%d", p, kMoeMaxRanks);
  if (cols == 0) return bad("cols is 0");
  if (cols > kNormMaxCols) return report_error(CCL_ERR_UNSUPPORTED, "cols=%zu above %zu", cols, kNormMaxCols);
  EXPERTS_TRY(check_float_dtype(dt, "rows"));
  EXPERTS_TRY(check_float_dtype(weight_dt, "weights"));
  if (rows == nullptr) return bad("rows is NULL");
  for (int r = 0; r < p; ++r)
    if (rows[r] > 0x7FFFFFFFull) return report_error(CCL_ERR_INVALID_ARG, "rows[%d] must stay below 2^31", r);
  return CCL_OK;
}

}  // namespace

extern "C" ccl_status_t ccl_layer_norm(const void* const* x, const void* const* residual, const void* const* weight,
                                       const void* const* bias, const size_t* rows, int p, size_t cols, double eps,
                                       ccl_dtype_t dt, ccl_dtype_t weight_dt, void* const* y, void* const* sum,
                                       float* const* mean, float* const* rstd, void* stream) {
  CCL_TRACE();
  clear_last_error();
  EXPERTS_TRY(check_norm(rows, p, cols, dt, weight_dt));
  if (!(isfinite(eps) && eps >= 0)) return bad("eps must be finite and not negative");
  if ((residual != nullptr) != (sum != nullptr)) return bad("residual and sum are given together");
  if ((mean != nullptr) != (rstd != nullptr)) return bad("mean and rstd are given together");
  if (!any_tokens(rows, p)) return CCL_OK;
  if (x == nullptr || weight == nullptr || y == nullptr) return bad("x, weight or y is NULL");
  const size_t e = dt == CCL_F32 ? 4 : 2, we = weight_dt == CCL_F32 ? 4 : 2;
  NormArgs a;
  NormSpans spans;
  memset(&a, 0, sizeof(a));
  uintptr_t bits = cols * e;
  for (int r = 0; r < p; ++r) {
    if (rows[r] == 0) continue;
    const uint64_t bytes = rows[r] * static_cast<uint64_t>(cols) * e;
    EXPERTS_TRY(check_buffer("x", r, x[r], e));
    EXPERTS_TRY(check_buffer("weight", r, weight[r], we));
    EXPERTS_TRY(check_buffer("y", r, y[r], e));
    a.x[r] = x[r];
    a.weight[r] = weight[r];
    a.out[r] = y[r];
    bits |= reinterpret_cast<uintptr_t>(x[r]) | reinterpret_cast<uintptr_t>(y[r]);
    spans.add(x[r], bytes, false);
    spans.add(weight[r], cols * we, false);
    spans.add(y[r], bytes, true);
    if (bias != nullptr) {
      EXPERTS_TRY(check_buffer("bias", r, bias[r], we));
      a.bias[r] = bias[r];
      spans.add(bias[r], cols * we, false);
    }
    if (residual != nullptr) {
      EXPERTS_TRY(check_buffer("residual", r, residual[r], e));
      EXPERTS_TRY(check_buffer("sum", r, sum[r], e));
      a.extra[r] = residual[r];
      a.sum[r] = sum[r];
      bits |= reinterpret_cast<uintptr_t>(residual[r]) | reinterpret_cast<uintptr_t>(sum[r]);
      spans.add(residual[r], bytes, false);
      spans.add(sum[r], bytes, true);
    }
    if (mean != nullptr) {
      EXPERTS_TRY(check_buffer("mean", r, mean[r], 4));
      EXPERTS_TRY(check_buffer("rstd", r, rstd[r], 4));
      a.mean[r] = mean[r];
      a.rstd[r] = rstd[r];
      spans.add(mean[r], rows[r] * 4, true);
      spans.add(rstd[r], rows[r] * 4, true);
    }
  }
  if (spans.clash()) return bad("an output overlaps another buffer");
  a.eps = eps;
  a.cols = static_cast<uint32_t>(cols);
  a.p = p;
  take_rows(&a.parts, rows, p);
  return launched(launch_norm(dt, weight_dt, on_grid(bits), &a, on(stream)), "layer norm kernel");
}

extern "C" size_t ccl_layer_norm_grad_workspace_bytes(int p, size_t cols) {
  if (p < 1 || p > kMoeMaxRanks || cols < 1 || cols > kNormMaxCols) return 0;
  return (kNormParts + static_cast<size_t>(p)) * 2 * cols * 4;
}

extern "C" ccl_status_t ccl_layer_norm_grad(const void* const* dy, const void* const* dsum, const void* const* x,
                                            const void* const* weight, const float* const* mean,
                                            const float* const* rstd, const size_t* rows, int p, size_t cols,
                                            ccl_dtype_t dt, ccl_dtype_t weight_dt, void* const* dx, ccl_dtype_t dw_dt,
                                            void* const* dweight, void* const* dbias, void* workspace,
                                            size_t workspace_bytes, void* stream) {
  CCL_TRACE();
  clear_last_error();
  EXPERTS_TRY(check_norm(rows, p, cols, dt, weight_dt));
  EXPERTS_TRY(check_float_dtype(dw_dt, "weight gradients"));
  const bool weights = dweight != nullptr || dbias != nullptr, any = any_tokens(rows, p);
  if (!weights && !any) return CCL_OK;
  if (any && (dy == nullptr || x == nullptr || weight == nullptr || mean == nullptr || rstd == nullptr || dx == nullptr))
    return bad("dy, x, weight, mean, rstd or dx is NULL");
  const size_t e = dt == CCL_F32 ? 4 : 2, we = weight_dt == CCL_F32 ? 4 : 2, de = dw_dt == CCL_F32 ? 4 : 2;
  NormArgs a;
  NormJoinArgs j;
  NormSpans spans;
  memset(&a, 0, sizeof(a));
  memset(&j, 0, sizeof(j));
  uintptr_t bits = cols * e;
  for (int r = 0; r < p; ++r) {
    if (dweight != nullptr) {
      EXPERTS_TRY(check_buffer("dweight", r, dweight[r], de));
      j.dweight[r] = dweight[r];
      spans.add(dweight[r], cols * de, true);
    }
    if (dbias != nullptr) {
      EXPERTS_TRY(check_buffer("dbias", r, dbias[r], de));
      j.dbias[r] = dbias[r];
      spans.add(dbias[r], cols * de, true);
    }
    if (rows[r] == 0) continue;
    const uint64_t bytes = rows[r] * static_cast<uint64_t>(cols) * e;
    EXPERTS_TRY(check_buffer("dy", r, dy[r], e));
    EXPERTS_TRY(check_buffer("x", r, x[r], e));
    EXPERTS_TRY(check_buffer("weight", r, weight[r], we));
    EXPERTS_TRY(check_buffer("mean", r, mean[r], 4));
    EXPERTS_TRY(check_buffer("rstd", r, rstd[r], 4));
    EXPERTS_TRY(check_buffer("dx", r, dx[r], e));
    a.dy[r] = dy[r];
    a.x[r] = x[r];
    a.weight[r] = weight[r];
    a.mean[r] = const_cast<float*>(mean[r]);  // read only
    a.rstd[r] = const_cast<float*>(rstd[r]);
    a.out[r] = dx[r];
    bits |= reinterpret_cast<uintptr_t>(dy[r]) | reinterpret_cast<uintptr_t>(x[r]) | reinterpret_cast<uintptr_t>(dx[r]);
    spans.add(dy[r], bytes, false);
    spans.add(x[r], bytes, false);
    spans.add(weight[r], cols * we, false);
    spans.add(mean[r], rows[r] * 4, false);
    spans.add(rstd[r], rows[r] * 4, false);
    spans.add(dx[r], bytes, true);
    if (dsum != nullptr) {
      EXPERTS_TRY(check_buffer("dsum", r, dsum[r], e));
      a.extra[r] = dsum[r];
      bits |= reinterpret_cast<uintptr_t>(dsum[r]);
      spans.add(dsum[r], bytes, false);
    }
  }
  if (weights) {
    const size_t need = ccl_layer_norm_grad_workspace_bytes(p, cols);
    if (workspace == nullptr || workspace_bytes < need)
      return report_error(CCL_ERR_INVALID_ARG, "workspace of %zu bytes needed", need);
    if (reinterpret_cast<uintptr_t>(workspace) & 15) return bad("workspace is not 16-byte aligned");
    spans.add(workspace, need, true);
  }
  if (spans.clash()) return bad("an output overlaps another buffer");
  a.partial = weights ? static_cast<float*>(workspace) : nullptr;  // one that is not needed has not been looked at
  a.cols = static_cast<uint32_t>(cols);
  a.p = p;
  take_rows(&a.parts, rows, p);
  if (any) EXPERTS_TRY(launched(launch_norm_grad(dt, weight_dt, on_grid(bits), &a, on(stream)), "layer norm gradient kernel"));
  if (!weights) return CCL_OK;
  memcpy(j.first, a.parts.first, sizeof(j.first));
  j.partial = a.partial;
  j.cols = a.cols;
  j.p = p;
  j.weight = dweight != nullptr;
  j.bias = dbias != nullptr;
  return launched(launch_norm_join(dw_dt, j, on(stream)), "layer norm sums kernel");
}
