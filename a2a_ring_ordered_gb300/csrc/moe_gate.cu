// moe_gate.cu -- the router's choice, its balance loss, and their gradients.
//
// A token's logits l, scores u (exp(l) or 1 / (1 + exp(-l))), shares p = u / sum u.
// The choice is the k largest logits; gates are u over the chosen ones' sum, or
// p, or u.  The loss is L = E / (k T^2) sum_e c_e sum_t p_te, c the counts.
// Scores are kept over a power of e so that the largest of a row stays away
// from 0: softmax over exp(max), sigmoid over exp(min(max, 0)).
#include "row_parts.cuh"

namespace ccl {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kWarps = kThreads / 32;

// Orders as the numbers do: -0 is 0, NaN comes last (the largest), -inf is 0.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __float_as_uint(l + 0.0f);
  if (l != l) return 0xFFFFFFFFu;
  if (l == -INFINITY) return 0;
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// u(l) over exp(base).
__device__ __forceinline__ float score_of(float l, float base, bool sigmoid) {
  return sigmoid ? expf(fminf(l, 0.f) - base) / (1.f + expf(-fabsf(l))) : expf(l - base);
}
// 1 - sigmoid(l)
__device__ __forceinline__ float away_of(float l) { return expf(-fmaxf(l, 0.f)) / (1.f + expf(-fabsf(l))); }
// The exponent of the power that a row's scores are kept over.
__device__ __forceinline__ float base_of(float top, bool sigmoid) {
  if (top == -INFINITY) return 0.f;
  return sigmoid ? fminf(top, 0.f) : top;
}

// A warp's row: column lane + 32 i in l[i], -inf behind the row.
template <int DT, int NV>
__device__ __forceinline__ void load_row(float* l, const void* base, uint64_t at, int experts, int lane) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 32 * i;
    l[i] = -INFINITY;
    if (e < experts) {
      if constexpr (DT == kF32) l[i] = static_cast<const float*>(base)[at + e];
      else l[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at + e]);
    }
  }
}

template <int DT, int NV, bool SELECT, bool BALANCE>
__global__ void __launch_bounds__(kThreads) gate_kernel(const __grid_constant__ GateArgs a) {
  extern __shared__ float shared[];  // BALANCE: [kWarps][E] sums of shares, then E + 1 counts
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.num_experts, k = a.k;
  const bool sigmoid = a.score == CCL_SCORE_SIGMOID;
  const RowPart part = row_part(a.parts, a.p, blockIdx.x);
  const int r = part.r;
  int* counts = reinterpret_cast<int*>(shared + kWarps * E);
  float sums[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) sums[i] = 0.f;
  if constexpr (BALANCE) {
    for (int i = threadIdx.x; i <= E; i += kThreads) counts[i] = 0;
    __syncthreads();
  }
  for (uint32_t row = part.lo + warp; row < part.hi; row += kWarps) {
    float l[NV];
    load_row<DT, NV>(l, a.logits[r], static_cast<uint64_t>(row) * E, E, lane);
    float top = l[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) top = fmaxf(top, l[i]);
    top = warp_max(top);
    bool live = false;
#pragma unroll
    for (int i = 0; i < NV; ++i) live |= !(l[i] == -INFINITY);
    live = __any_sync(kAll, live);
    const float base = base_of(top, sigmoid);
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) total += score_of(l[i], base, sigmoid);
    total = warp_sum(total);
    const uint64_t item = static_cast<uint64_t>(row) * k + lane;
    int id = -1;
    if constexpr (SELECT) {
      uint32_t key[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] = lane + 32 * i < E ? key_of(l[i]) : 0;
      float chosen = 0.f;
      for (int j = 0; j < k; ++j) {
        uint32_t best = 0;
        int at = 0;
        float value = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (key[i] > best) {
            best = key[i];
            at = lane + 32 * i;
            value = l[i];
          }
        const uint32_t most = __reduce_max_sync(kAll, best);
        const uint32_t first = __reduce_min_sync(kAll, best == most ? at : 0x7FFFFFFF);
        value = __shfl_sync(kAll, value, first & 31);
        if (lane == j && most != 0) {
          id = static_cast<int>(first);
          chosen = value;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (most != 0 && lane + 32 * i == static_cast<int>(first)) key[i] = 0;
      }
      if (a.normalize || !sigmoid) {
        const float u = id >= 0 ? score_of(chosen, base, sigmoid) : 0.f;
        const float over = a.normalize ? warp_sum(u) : total;
        chosen = over == 0.f ? 0.f : u / over;
      } else {
        chosen = score_of(chosen, 0.f, true);
      }
      if (lane < k) {
        a.ids[r][item] = id;
        a.gates[r][item] = id >= 0 ? a.scale * chosen : 0.f;
      }
    } else if (lane < k) {
      id = a.ids_in[r][item];
    }
    if constexpr (BALANCE) {
      if (id >= 0 && id < E) atomicAdd(counts + id, 1);
      if (lane == 0 && live) atomicAdd(counts + E, 1);
      if (total != 0.f) {
#pragma unroll
        for (int i = 0; i < NV; ++i) sums[i] += score_of(l[i], base, sigmoid) / total;
      }
    }
  }
  if (!BALANCE) return;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (lane + 32 * i < E) shared[warp * E + lane + 32 * i] = sums[i];
  __syncthreads();
  float* out = a.partial + blockIdx.x * balance_part_words(E);
  for (int e = threadIdx.x; e <= E; e += kThreads) {
    if (e < E) {
      float s = 0.f;
      for (int w = 0; w < kWarps; ++w) s += shared[w * E + e];
      out[e] = s;
    }
    reinterpret_cast<int*>(out)[E + e] = counts[e];
  }
}

// One CTA per rank adds up the parts of its own, or of all where the ranks'
// tokens are one batch.
__global__ void __launch_bounds__(kThreads) balance_join_kernel(const __grid_constant__ BalanceJoinArgs a) {
  __shared__ double warp_sums[kWarps];
  pdl_enter();
  const int r = blockIdx.x, E = a.num_experts;
  const uint32_t lo = a.together ? 0 : a.first[r], hi = a.together ? a.first[a.p] : a.first[r + 1];
  const size_t words = balance_part_words(E);
  double sum = 0.0;
  for (int e = threadIdx.x; e < E; e += kThreads) {
    double s = 0.0;
    int c = 0;
    for (uint32_t i = lo; i < hi; ++i) {
      s += a.partial[i * words + e];
      c += reinterpret_cast<const int*>(a.partial)[i * words + E + e];
    }
    a.counts[r][e] = c;
    sum += s * c;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x != 0) return;
  sum = 0.0;
  for (int w = 0; w < kWarps; ++w) sum += warp_sums[w];
  int t = 0;
  for (uint32_t i = lo; i < hi; ++i) t += reinterpret_cast<const int*>(a.partial)[i * words + 2 * E];
  a.counts[r][E] = t;
  a.losses[r][0] = t == 0 ? 0.f : static_cast<float>(sum * E / (static_cast<double>(a.k) * t * t));
}

template <int DT, int NV, bool GATES, bool BALANCE>
__global__ void __launch_bounds__(kThreads) gate_grad_kernel(const __grid_constant__ GateArgs a) {
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.num_experts, k = a.k;
  const bool sigmoid = a.score == CCL_SCORE_SIGMOID;
  const RowPart part = row_part(a.parts, a.p, blockIdx.x);
  const int r = part.r;
  float weight[NV];  // of the loss: E / (k T^2) (c_e - mean c) dloss; a constant taken off changes nothing
  if constexpr (BALANCE) {
    const int* counts = a.counts[r];
    int64_t all = 0;
    for (int e = lane; e < E; e += 32) all += counts[e];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(kAll, all, o);
    const double t = counts[E] > 0 ? counts[E] : 1.0;
    const double d = static_cast<double>(a.dlosses[r] != nullptr ? a.dlosses[r][0] : 1.f) * a.balance_scale * E / (k * t * t);
    const double mean = static_cast<double>(all) / E;
#pragma unroll
    for (int i = 0; i < NV; ++i) weight[i] = lane + 32 * i < E ? static_cast<float>(d * (counts[lane + 32 * i] - mean)) : 0.f;
  }
  for (uint32_t row = part.lo + warp; row < part.hi; row += kWarps) {
    const uint64_t at = static_cast<uint64_t>(row) * E;
    float l[NV], out[NV];
    load_row<DT, NV>(l, a.logits[r], at, E, lane);
    float top = l[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) top = fmaxf(top, l[i]);
    top = warp_max(top);
    const float base = base_of(top, sigmoid);
    float share[NV], total = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) total += share[i] = score_of(l[i], base, sigmoid);
    total = warp_sum(total);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      share[i] = total == 0.f ? 0.f : share[i] / total;
      out[i] = 0.f;
    }
    if constexpr (BALANCE) {
      float mean = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) mean += share[i] * weight[i];
      mean = warp_sum(mean);
#pragma unroll
      for (int i = 0; i < NV; ++i) out[i] = share[i] * (weight[i] - mean);
    }
    if constexpr (GATES) {
      int id = -1;
      float d = 0.f, value = 0.f;
      if (lane < k) {
        id = a.ids_in[r][static_cast<uint64_t>(row) * k + lane];
        if (id < 0 || id >= E) id = -1;
      }
      if (id >= 0) {
        d = a.scale * a.dgates[r][static_cast<uint64_t>(row) * k + lane];
        if constexpr (DT == kF32) value = static_cast<const float*>(a.logits[r])[at + id];
        else value = __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits[r])[at + id]);
      }
      // what a choice adds to its expert's gradient, and every expert's part of the softmax's
      float own = 0.f, all = 0.f;
      if (a.normalize) {
        const float u = id >= 0 ? score_of(value, base, sigmoid) : 0.f;
        const float over = warp_sum(u), g = over == 0.f ? 0.f : u / over;
        const float mean = warp_sum(g * d);
        own = g * (d - mean);
      } else if (sigmoid) {
        own = id >= 0 ? score_of(value, 0.f, true) * d : 0.f;
      } else {
        own = id >= 0 && total != 0.f ? score_of(value, base, false) / total * d : 0.f;
        all = warp_sum(own);
      }
      float into[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) into[i] = 0.f;
      for (int j = 0; j < k; ++j) {
        const int e = __shfl_sync(kAll, id, j);
        const float v = __shfl_sync(kAll, own, j);
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (lane + 32 * i == e) into[i] += v;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) out[i] += into[i] - share[i] * all;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 32 * i;
      if (e >= E) continue;
      const float v = sigmoid ? out[i] * away_of(l[i]) : out[i];
      if constexpr (DT == kF32) static_cast<float*>(a.dlogits[r])[at + e] = v;
      else static_cast<__nv_bfloat16*>(a.dlogits[r])[at + e] = __float2bfloat16_rn(v);
    }
  }
}

// Calls f(DT, NV) with the values a lane holds.
template <typename F>
cudaError_t by_width(int dt, int experts, F f) {
  const auto with = [&](auto d) {
    if (experts <= 32) return f(d, std::integral_constant<int, 1>{});
    if (experts <= 64) return f(d, std::integral_constant<int, 2>{});
    if (experts <= 128) return f(d, std::integral_constant<int, 4>{});
    if (experts <= 256) return f(d, std::integral_constant<int, 8>{});
    if (experts <= 512) return f(d, std::integral_constant<int, 16>{});
    return f(d, std::integral_constant<int, 32>{});
  };
  return dt == kF32 ? with(std::integral_constant<int, kF32>{}) : with(std::integral_constant<int, kBF16>{});
}

cudaError_t launch_parts(void (*kernel)(GateArgs), const GateArgs& a, size_t smem, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.parts.first[a.p]);
  cfg.blockDim = dim3(kThreads);
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

}  // namespace

cudaError_t launch_gate(int dt, bool, bool select, bool balance, const GateArgs& a, cudaStream_t s) {
  const size_t smem = balance ? (static_cast<size_t>(kWarps) * a.num_experts + a.num_experts + 1) * 4 : 0;
  return by_width(dt, a.num_experts, [&](auto d, auto nv) {
    constexpr int DT = decltype(d)::value, NV = decltype(nv)::value;
    return launch_parts(!select ? gate_kernel<DT, NV, false, true> : balance ? gate_kernel<DT, NV, true, true> : gate_kernel<DT, NV, true, false>,
                        a, smem, s);
  });
}

cudaError_t launch_balance_join(const BalanceJoinArgs& a, cudaStream_t s) {
  const cudaError_t err = launch_kernel(balance_join_kernel, dim3(static_cast<unsigned>(a.p)), dim3(kThreads), s, a);
  if (err == cudaSuccess) note_launch();
  return err;
}

cudaError_t launch_gate_grad(int dt, bool, bool gates, bool balance, const GateArgs& a, cudaStream_t s) {
  return by_width(dt, a.num_experts, [&](auto d, auto nv) {
    constexpr int DT = decltype(d)::value, NV = decltype(nv)::value;
    return launch_parts(!gates ? gate_grad_kernel<DT, NV, false, true> : balance ? gate_grad_kernel<DT, NV, true, true> : gate_grad_kernel<DT, NV, true, false>,
                        a, 0, s);
  });
}

}  // namespace ccl
