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
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr (L == 32) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(m) : "f"(v));  // as fmaxf: numbers before NaN
    return m;
  } else {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAllLanes, v, o));
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
// exp(l - base) is the hardware's power of two of the rounded (l - base) log2(e):
// off by |l - base| 2^-23 and two units more, which gates and shares, of fp32,
// carry on.  (One fused multiply-add would do for both, but base log2(e) is not
// finite where a row is masked by the type's lowest value.)
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float power_of_two(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float reciprocal_of(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
__device__ __forceinline__ float base_of(float top, bool sigmoid) {
  if (top == -INFINITY) return 0.f;
  return sigmoid ? fminf(top, 0.f) : top;
}
__device__ __forceinline__ float softmax_score(float l, float base) { return power_of_two((l - base) * kLog2e); }
// u, and 1 - sigmoid(l), of one logit; base is 0 for nearly every row.
struct Sigmoid {
  float t, r;  // exp(-|l|), 1 / (1 + t)
  __device__ __forceinline__ explicit Sigmoid(float l) : t(power_of_two(-fabsf(l) * kLog2e)), r(reciprocal_of(1.f + t)) {}
  __device__ __forceinline__ float score(float l) const { return l >= 0.f ? r : t * r; }
  __device__ __forceinline__ float score(float l, float base) const { return base == 0.f ? score(l) : softmax_score(fminf(l, 0.f), base) * r; }
  __device__ __forceinline__ float away(float l) const { return l > 0.f ? t * r : r; }
};
__device__ __forceinline__ float sigmoid_score(float l, float base) { return Sigmoid(l).score(l, base); }
__device__ __forceinline__ float score_of(float l, float base, bool sigmoid) { return sigmoid ? sigmoid_score(l, base) : softmax_score(l, base); }
// All scores of a lane's columns, in pairs, and their sum; AWAY: and 1 - sigmoid.
template <int DT, int NV, bool AWAY>
__device__ __forceinline__ float scores_of(const GateRow<DT, NV>& row, float base, bool sigmoid, F2* u, F2* away) {
  F2 sum = both(0.f);
  if (sigmoid) {
#pragma unroll
    for (int k = 0; k < NV / 2; ++k) {
      const float x = row.value(2 * k), y = row.value(2 * k + 1);
      const Sigmoid a(x), b(y);
      u[k] = pair(a.score(x), b.score(y));
      if constexpr (AWAY) away[k] = pair(a.away(x), b.away(y));
    }
    if (base != 0.f) {
#pragma unroll
      for (int k = 0; k < NV / 2; ++k) u[k] = pair(sigmoid_score(row.value(2 * k), base), sigmoid_score(row.value(2 * k + 1), base));
    }
  } else {
    const F2 scale = both(kLog2e), less = both(-base);
#pragma unroll
    for (int k = 0; k < NV / 2; ++k) {
      const float2 x = parts(mul2(add2(pair(row.value(2 * k), row.value(2 * k + 1)), less), scale));
      u[k] = pair(power_of_two(x.x), power_of_two(x.y));
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
