// api_checks.h -- argument checks shared by the entry points of a rank's own
// layer work (experts, router, norm, AdamW).  Host code only.
#pragma once

#include <algorithm>

#include "ccl_internal.h"

namespace ccl {

#define EXPERTS_TRY(call)                    \
  do {                                       \
    const ccl_status_t st_ = (call);         \
    if (st_ != CCL_OK) return st_;           \
  } while (0)

inline ccl_status_t bad(const char* what) { return report_error(CCL_ERR_INVALID_ARG, "%s", what); }

// The byte ranges of a call: an output may overlap nothing.  Fixed storage,
// so that no entry point can throw.
template <int CAP>
class SpansOf {
 public:
  void add(const void* p, uint64_t bytes, bool out) {
    if (bytes == 0 || p == nullptr) return;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    s_[n_++] = {lo, lo + bytes, out};
  }
  bool clash() {
    std::sort(s_, s_ + n_, [](const Span& a, const Span& b) { return a.lo < b.lo; });
    uintptr_t any = 0, out = 0;  // furthest end so far, of all and of outputs
    for (int i = 0; i < n_; ++i) {
      if (s_[i].lo < out || (s_[i].out && s_[i].lo < any)) return true;
      any = std::max(any, s_[i].hi);
      if (s_[i].out) out = std::max(out, s_[i].hi);
    }
    return false;
  }

 private:
  struct Span {
    uintptr_t lo, hi;
    bool out;
  };
  Span s_[CAP];
  int n_ = 0;
};

inline ccl_status_t check_buffer(const char* name, int r, const void* p, size_t align) {
  if (p == nullptr) return report_error(CCL_ERR_INVALID_ARG, "%s[%d] is NULL", name, r);
  if (reinterpret_cast<uintptr_t>(p) % align)
    return report_error(CCL_ERR_INVALID_ARG, "%s[%d] is not %zu-byte aligned", name, r, align);
  return CCL_OK;
}

// p ranks, k choices and the tokens of each rank.
inline ccl_status_t check_tokens(const size_t* tokens, int p, int k) {
  if (p < 1 || p > kMoeMaxRanks) return report_error(CCL_ERR_INVALID_ARG, "p=%d outside 1..%d", p, kMoeMaxRanks);
  if (k < 1 || k > kMoeMaxK) return report_error(CCL_ERR_INVALID_ARG, "k=%d outside 1..%d", k, kMoeMaxK);
  if (tokens == nullptr) return bad("tokens is NULL");
  for (int r = 0; r < p; ++r)
    if (tokens[r] > 0x7FFFFFFFull / static_cast<size_t>(k))
      return report_error(CCL_ERR_INVALID_ARG, "tokens[%d] * k must stay below 2^31", r);
  return CCL_OK;
}

inline ccl_status_t check_float_dtype(ccl_dtype_t dt, const char* what) {
  if (dt != CCL_F32 && dt != CCL_BF16)
    return dt == CCL_I32 ? report_error(CCL_ERR_UNSUPPORTED, "%s are fp32 or bf16", what)
                         : report_error(CCL_ERR_INVALID_ARG, "unknown dtype %d", static_cast<int>(dt));
  return CCL_OK;
}

inline bool any_tokens(const size_t* tokens, int p) {
  for (int r = 0; r < p; ++r)
    if (tokens[r] != 0) return true;
  return false;
}

// Whether all rows start on 16 bytes; `bits`: addresses and row bytes or-ed together.
inline bool on_grid(uintptr_t bits) { return (bits & 15) == 0; }

inline ccl_status_t launched(cudaError_t err, const char* what) {
  if (err == cudaSuccess) return CCL_OK;
  return report_error(CCL_ERR_CUDA, "%s launch: %s (%s)", what, cudaGetErrorString(err), cudaGetErrorName(err));
}

inline cudaStream_t on(void* stream) { return static_cast<cudaStream_t>(stream); }

}  // namespace ccl
