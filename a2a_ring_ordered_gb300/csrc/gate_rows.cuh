// gate_rows.cuh -- a token's logits in the registers of a few lanes, shared by
// the router's kernels.
//
// L lanes (a power of two), a team, have a row, NV columns each: eight consecutive ones at
// lane * 8, and where a row has more than 256 columns again at 256, 512, ... of
// them.  So a lane's columns come by 16-byte loads, and of equal logits the
// lowest lane has the lowest column.  Columns behind the row are -inf.
#pragma once

#include "pairs.cuh"
#include "row_parts.cuh"

namespace ccl {

constexpr unsigned kAllLanes = 0xFFFFFFFFu;

template <int L>
__device__ __forceinline__ int gate_column(int lane, int i) {
  return (i / 8) * (8 * L) + lane * 8 + i % 8;
}

template <int DT, int NV>
struct GateRow {
  static constexpr int kWords = NV * Elem<DT>::kBytes / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ float value(int i) const { return widen<DT>(w, i); }

  // `there`: the row exists; `vec`: rows start on 16 bytes.
  template <int L>
  __device__ __forceinline__ void load(const void* logits, uint64_t row, int experts, int lane, bool there, bool vec) {
    constexpr uint32_t kNone = DT == kF32 ? 0xFF800000u : 0xFF80FF80u;  // -inf
    constexpr int kPer = 16 / Elem<DT>::kBytes;
    const char* base = static_cast<const char*>(logits) + row * experts * Elem<DT>::kBytes;
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = kNone;
    if (!there) return;
    if (vec) {
#pragma unroll
      for (int q = 0; q < NV / kPer; ++q) {
        const int c = gate_column<L>(lane, q * kPer);
        if (c >= experts) continue;
        const uint4 v = ld_l1_16(base + c * Elem<DT>::kBytes);
        w[4 * q] = v.x;
        w[4 * q + 1] = v.y;
        w[4 * q + 2] = v.z;
        w[4 * q + 3] = v.w;
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = gate_column<L>(lane, i);
      if (c >= experts) continue;
      if constexpr (DT == kF32) {
        w[i] = __ldg(reinterpret_cast<const uint32_t*>(base) + c);
      } else {
        const uint32_t h = __ldg(reinterpret_cast<const unsigned short*>(base) + c);
        w[i / 2] = (i & 1) ? (w[i / 2] & 0xFFFFu) | h << 16 : (w[i / 2] & 0xFFFF0000u) | h;
      }
    }
  }
};

template <int DT>
__device__ __forceinline__ float gate_logit(const void* logits, uint64_t row, int experts, int e) {
  const uint64_t at = row * experts + e;
  if constexpr (DT == kF32) return __ldg(static_cast<const float*>(logits) + at);
  else return __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const unsigned short*>(logits) + at)) << 16);
}

// A row's choices have C lanes, so that a warp, which has 32 / L rows at a time,
// settles the choices of 32 / C rows at once: a batch, of L / C passes.  In pass j a
// team has the batch's row team * L / C + j, whose choices are in lanes j C .. of the
// team.  KM: the most choices.
template <int L, int KM>
struct GateBatch {
  static constexpr int kChoices = L < KM ? L : KM, kRows = 32 / kChoices, kPasses = L / kChoices;
};

// ------------------------------------------------------------ among L lanes
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAllLanes, v, o);
  return v;
}
// Two sums by the shuffles of little more than one: half of the lanes take each.
template <int L>
__device__ __forceinline__ float2 lanes_sum(float a, float b) {
  if constexpr (L == 1) {
    return make_float2(a, b);
  } else {
    const bool upper = (threadIdx.x & (L / 2)) != 0;
    float v = (upper ? b : a) + __shfl_xor_sync(kAllLanes, upper ? a : b, L / 2);
#pragma unroll
    for (int o = L / 4; o > 0; o >>= 1) v += __shfl_xor_sync(kAllLanes, v, o);
    return make_float2(__shfl_sync(kAllLanes, v, 0, L), __shfl_sync(kAllLanes, v, L / 2, L));
  }
}
// Of two numbers; NaN where one of them is.
__device__ __forceinline__ float larger(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}
__device__ __forceinline__ float smaller(float a, float b) {
  float m;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr (L == 32) {
    float m;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xFFFFFFFF;" : "=f"(m) : "f"(v));
    return m;
  } else {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = larger(v, __shfl_xor_sync(kAllLanes, v, o));
    return v;
  }
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  if constexpr (L == 32) {
    return __reduce_max_sync(kAllLanes, v);
  } else {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kAllLanes, v, o));
    return v;
  }
}
template <int L>
__device__ __forceinline__ uint32_t lanes_min(uint32_t v) {
  if constexpr (L == 32) {
    return __reduce_min_sync(kAllLanes, v);
  } else {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(kAllLanes, v, o));
    return v;
  }
}

// ------------------------------------------------------------------- scores
// Scores are kept over exp(base), base max(row) for softmax and min(max(row), 0)
// for sigmoid, so that the row's largest stays away from 0; 0 for a row of -inf.
//
// exp(x) of x = l - base <= 0 is the hardware's power of two of t = x log2(e), which
// is rounded: by itself that is off by |x| 2^-23, and so is a gate or a share of a
// logit far from its row's top.  Times 1 + r, r = x - t ln 2 (below 2^-16) being what
// the rounding left, it is off by some four roundings of 2^-24, and |x| 2^-28 more
// because ln 2 is rounded too.  A sum of scores goes without: by the weight of the
// scores in it, the mean of |x| is at most the logarithm of their number.
//
// (One fused multiply-add would do for x and t both, but base log2(e) is not finite
// where a row is masked by the type's lowest value.)
constexpr float kLog2e = static_cast<float>(1.4426950408889634), kLn2 = static_cast<float>(0.6931471805599453);
__device__ __forceinline__ float power_of_two(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rough_exp(float x) { return power_of_two(x * kLog2e); }
__device__ __forceinline__ F2 rough_exp(F2 x) {
  const float2 t = parts(mul2(x, both(kLog2e)));
  return pair(power_of_two(t.x), power_of_two(t.y));
}
__device__ __forceinline__ float exp_of(float x) {
  x = larger(x, -128.f);  // -inf has no r; NaN stays
  const float t = __fmul_rn(x, kLog2e), y = power_of_two(t);
  return fmaf(y, fmaf(t, -kLn2, x), y);
}
// a b + c within 0 and 1, NaN as 0.
__device__ __forceinline__ float fma_sat(float a, float b, float c) {
  float d;
  asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Of a row's columns: 0 for -inf, and for a NaN too, of which the row's base tells.
__device__ __forceinline__ F2 exp_of(F2 x) {
  const F2 t = mul2(x, both(kLog2e));
  const float2 e = parts(t), r = parts(fma2(t, both(-kLn2), x));
  const float a = power_of_two(e.x), b = power_of_two(e.y);
  return pair(fma_sat(a, r.x, a), fma_sat(b, r.y, b));
}
__device__ __forceinline__ float rough_reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// That, and a step of Newton's method.
__device__ __forceinline__ float reciprocal_of(float x) {
  const float y = rough_reciprocal(x);
  return fmaf(fmaf(-x, y, 1.f), y, y);
}
// u / v by Markstein's correction of the quotient: u / u is 1 to the bit.
__device__ __forceinline__ float quotient(float u, float v, float inv) {
  const float q = u * inv;
  return fmaf(fmaf(-q, v, u), inv, q);
}
__device__ __forceinline__ F2 quotient(F2 u, float v, F2 inv) {
  const F2 q = mul2(u, inv);
  return fma2(fma2(q, both(-v), u), inv, q);
}
// NaN where the row has one (sigmoid: where its largest is one).
__device__ __forceinline__ float base_of(float top, bool sigmoid) {
  if (top == -INFINITY) return 0.f;
  return sigmoid ? smaller(top, 0.f) : top;
}
__device__ __forceinline__ float softmax_score(float l, float base) { return exp_of(l - base); }
// u, and 1 - sigmoid(l), of one logit; base is 0 for nearly every row.
struct Sigmoid {
  float t, r;  // exp(-|l|), 1 / (1 + t)
  __device__ __forceinline__ Sigmoid(float t, float r) : t(t), r(r) {}
  __device__ __forceinline__ explicit Sigmoid(float l) : t(exp_of(-fabsf(l))), r(reciprocal_of(1.f + t)) {}
  __device__ __forceinline__ float score(float l) const { return l >= 0.f ? r : t * r; }
  __device__ __forceinline__ float score(float l, float base) const { return base == 0.f ? score(l) : softmax_score(fminf(l, 0.f), base) * r; }
  __device__ __forceinline__ float away(float l) const { return l > 0.f ? t * r : r; }
};
// Of two, of a row.
struct Sigmoids {
  Sigmoid a, b;
};
template <bool EACH>
__device__ __forceinline__ Sigmoids sigmoids(float x, float y) {
  float2 t;
  if constexpr (EACH) t = parts(exp_of(pair(-fabsf(x), -fabsf(y))));
  else t = make_float2(rough_exp(-fabsf(x)), rough_exp(-fabsf(y)));
  return {Sigmoid(t.x, rough_reciprocal(1.f + t.x)), Sigmoid(t.y, rough_reciprocal(1.f + t.y))};
}
__device__ __forceinline__ float sigmoid_score(float l, float base) { return Sigmoid(l).score(l, base); }
__device__ __forceinline__ float score_of(float l, float base, bool sigmoid) { return sigmoid ? sigmoid_score(l, base) : softmax_score(l, base); }
// A score of a row whose logits are all below 0.
template <bool EACH>
__device__ __forceinline__ float far_sigmoid(float l, float base) {
  if constexpr (EACH) return sigmoid_score(l, base);
  else return rough_exp(fminf(l, 0.f) - base) * rough_reciprocal(1.f + rough_exp(-fabsf(l)));
}
// All scores of a lane's columns, in pairs, and their sum.  EACH: each is wanted as it is,
// not the sum alone; AWAY: and 1 - sigmoid.
template <int DT, int NV, bool EACH, bool AWAY>
__device__ __forceinline__ float scores_of(const GateRow<DT, NV>& row, float base, bool sigmoid, F2* u, F2* away) {
  F2 sum = pair(EACH ? base - base : 0.f, 0.f);  // NaN where the base is
  if (sigmoid) {
#pragma unroll
    for (int k = 0; k < NV / 2; ++k) {
      const float x = row.value(2 * k), y = row.value(2 * k + 1);
      const Sigmoids v = sigmoids<EACH>(x, y);
      u[k] = pair(v.a.score(x), v.b.score(y));
      if constexpr (AWAY) away[k] = pair(v.a.away(x), v.b.away(y));
    }
    if (base != 0.f) {
#pragma unroll
      for (int k = 0; k < NV / 2; ++k) u[k] = pair(far_sigmoid<EACH>(row.value(2 * k), base), far_sigmoid<EACH>(row.value(2 * k + 1), base));
    }
  } else {
    const F2 less = both(-base);
#pragma unroll
    for (int k = 0; k < NV / 2; ++k) {
      const F2 x = add2(pair(row.value(2 * k), row.value(2 * k + 1)), less);
      if constexpr (EACH) u[k] = exp_of(x);
      else u[k] = rough_exp(x);
    }
  }
#pragma unroll
  for (int k = 0; k < NV / 2; ++k) sum = add2(sum, u[k]);
  return total2(sum);
}

// Lanes of a row that can hold the choices and, eight columns each, the row.
inline int gate_lanes(int experts, int k) {
  int lanes = 1;
  while (lanes < 32 && (lanes * 8 < experts || lanes < k)) lanes *= 2;
  return lanes;
}

// Calls f(DT, L, NV).
template <typename F>
cudaError_t by_row(int dt, int experts, int k, F f) {
  const auto with = [&](auto d) {
    constexpr std::integral_constant<int, 8> eight{};
    if (experts > 512) return f(d, std::integral_constant<int, 32>{}, std::integral_constant<int, 32>{});
    if (experts > 256) return f(d, std::integral_constant<int, 32>{}, std::integral_constant<int, 16>{});
    switch (gate_lanes(experts, k)) {
      case 1: return f(d, std::integral_constant<int, 1>{}, eight);
      case 2: return f(d, std::integral_constant<int, 2>{}, eight);
      case 4: return f(d, std::integral_constant<int, 4>{}, eight);
      case 8: return f(d, std::integral_constant<int, 8>{}, eight);
      case 16: return f(d, std::integral_constant<int, 16>{}, eight);
      default: return f(d, std::integral_constant<int, 32>{}, eight);
    }
  };
  return dt == kF32 ? with(std::integral_constant<int, kF32>{}) : with(std::integral_constant<int, kBF16>{});
}

inline cudaError_t launch_gate_parts(void (*kernel)(GateArgs), const GateArgs& a, int threads, size_t smem, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.parts.first[a.p]);
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = CCL_PDL ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, a);
  if (err == cudaSuccess) note_launch();
  return err;
}

}  // namespace ccl
