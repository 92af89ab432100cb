// moe_gate_grad.cu -- the gradients of the router's gates and of its balance
// loss for the logits.
//
// With p the shares, g the gates, d = dgates and a_e = dloss E / (k T^2) c_e:
//   loss:                    p_e (a_e - sum a p)
//   gates, normalised:       g_e (d_e - sum d g / scale), for the chosen
//   gates, softmax:          g_e d_e for the chosen, - p_e sum d g for all
//   gates, sigmoid:          g_e d_e, for the chosen
// and all of it times 1 - sigmoid(l_e) for sigmoid scores.
//
// Logits are read once and gradients written once: HBM bounds it.
#include "gate_rows.cuh"

namespace ccl {
namespace {

template <int DT, int L, int NV, bool GATES, bool BALANCE>
__global__ void __launch_bounds__(kThreads) gate_grad_kernel(const __grid_constant__ GateArgs a) {
  constexpr int kRows = 32 / L, kWarps = kThreads / 32;
  // GATES: per warp, what the choices of its rows add to their columns; zeros between rows
  __shared__ __align__(16) float spread[GATES ? kWarps * 32 * NV : 1];
  __shared__ float unit;
  __shared__ int mean_count, mean_rest;  // sum c = E mean_count + mean_rest
  pdl_enter();
  const int lane = threadIdx.x & (L - 1), warp = threadIdx.x >> 5, team = (threadIdx.x & 31) / L, E = a.num_experts, k = a.k;
  const bool sigmoid = a.score == CCL_SCORE_SIGMOID, vec = a.vec != 0;
  // whether every column has a gradient, or the chosen ones alone
  const bool dense = BALANCE || !(a.normalize || sigmoid);
  const RowPart part = row_part(a.parts, a.p, blockIdx.x);
  const int r = part.r;
  float* mine = spread + (warp * kRows + team) * (L * NV);
  if constexpr (GATES) {
    for (int i = threadIdx.x & 31; i < 32 * NV; i += 32) spread[warp * 32 * NV + i] = 0.f;
    __syncwarp();
  }
  F2 weight[NV / 2];  // a_e, less a constant that changes nothing: counts near one another do not cancel
  if constexpr (BALANCE) {
    const int* counts = a.counts[r];
    if (warp == 0) {
      long long all = 0;
      for (int e = threadIdx.x; e < E; e += 32) all += counts[e];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(kAllLanes, all, o);
      if (threadIdx.x == 0) {
        mean_count = static_cast<int>(all / E);
        mean_rest = static_cast<int>(all - static_cast<long long>(mean_count) * E);
        const float t = counts[E] > 0 ? static_cast<float>(counts[E]) : 1.f;
        unit = (a.dlosses[r] != nullptr ? a.dlosses[r][0] : 1.f) * a.balance_scale / t / (t * k);
      }
    }
    __syncthreads();
    // E c_e - sum c, times dloss / (k T^2)
    const auto of = [&](int e) { return e < E ? fmaf(static_cast<float>(counts[e] - mean_count), static_cast<float>(E), -static_cast<float>(mean_rest)) * unit : 0.f; };
#pragma unroll
    for (int i = 0; i < NV; i += 2) weight[i / 2] = pair(of(gate_column<L>(lane, i)), of(gate_column<L>(lane, i + 1)));
  }
  uint64_t row0 = part.lo + static_cast<uint64_t>(warp) * kRows;
  GateRow<DT, NV> next;
  next.template load<L>(a.logits[r], row0 + team, E, lane, row0 + team < part.hi, vec);
  int next_id = -1;
  float next_d = 0.f;
  const auto fetch_choice = [&](uint64_t row) {
    next_id = -1;
    next_d = 0.f;
    if (lane < k && row < part.hi) {
      next_id = a.ids_in[r][row * k + lane];
      next_d = a.dgates[r][row * k + lane];
    }
  };
  if constexpr (GATES) fetch_choice(row0 + team);
  for (; row0 < part.hi; row0 += kWarps * kRows) {
    const uint64_t row = row0 + team, ahead = row + kWarps * kRows;
    const bool there = row < part.hi;
    const GateRow<DT, NV> now = next;
    int id = next_id;
    float d = a.scale * next_d;
    next.template load<L>(a.logits[r], ahead, E, lane, ahead < part.hi, vec);
    if constexpr (GATES) fetch_choice(ahead);
    if (id < 0 || id >= E) {
      id = -1;
      d = 0.f;  // whatever stands there
    }
    float value = -INFINITY;
    if (GATES && id >= 0) value = gate_logit<DT>(a.logits[r], row, E, id);
    F2 out[NV / 2], away[NV / 2];
    float total = 0.f, inv = 0.f, base = 0.f;
    if (dense) {
      float top = now.value(0);
#pragma unroll
      for (int i = 1; i < NV; ++i) top = fmaxf(top, now.value(i));
      base = base_of(lanes_max<L>(top), sigmoid);
      total = lanes_sum<L>(scores_of<DT, NV, true>(now, base, sigmoid, out, away));
      inv = total == 0.f ? 0.f : reciprocal_of(total);
    }
    float own = 0.f, all = 0.f;  // what this lane's choice adds to its column, and to all columns by their shares
    if constexpr (GATES) {
      constexpr int kMost = L < kMoeMaxK ? L : kMoeMaxK;  // no choices behind them
      if (a.normalize) {
        // over the chosen ones' largest, which may be far below the row's
        const float chosen_base = base_of(lanes_max<kMost>(value), sigmoid), u = id >= 0 ? score_of(value, chosen_base, sigmoid) : 0.f;
        const float over = lanes_sum<kMost>(u), g = over == 0.f ? 0.f : quotient(u, over, reciprocal_of(over));
        const float mean = lanes_sum<kMost>(g * d);
        own = g * (d - mean);
      } else {
        if (id >= 0) own = sigmoid ? sigmoid_score(value, 0.f) * d : quotient(softmax_score(value, base), total, inv) * d;
        if (!sigmoid) all = lanes_sum<L>(own);
      }
    }
    if (dense) {
      // shares; a lone one is 1 to the bit, so that it has no gradient
      F2 mean2 = both(0.f);
#pragma unroll
      for (int i = 0; i < NV / 2; ++i) {
        out[i] = quotient(out[i], total, both(inv));
        if constexpr (BALANCE) mean2 = fma2(out[i], weight[i], mean2);
      }
      float less = all;
      if constexpr (BALANCE) less += lanes_sum<L>(total2(mean2));
#pragma unroll
      for (int i = 0; i < NV / 2; ++i) {
        if constexpr (BALANCE) out[i] = mul2(out[i], add2(weight[i], both(-less)));
        else out[i] = mul2(out[i], both(-less));
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV / 2; ++i) out[i] = both(0.f);
    }
    if constexpr (GATES) {
      // an expert that the token has twice is added up by the one of its lanes whose number stands there in the end
      if (id >= 0) mine[id] = __int_as_float(lane);
      __syncwarp();
      const bool first = id >= 0 && __float_as_int(mine[id]) == lane;
      if (__any_sync(kAllLanes, id >= 0 && !first)) {
        float s = 0.f;
        for (int q = 0; q < L && q < k; ++q) {
          const float v = __shfl_sync(kAllLanes, own, q, L);
          if (__shfl_sync(kAllLanes, id, q, L) == id) s += v;
        }
        own = s;
      }
      __syncwarp();
      if (first) mine[id] = own;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < NV; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(mine + gate_column<L>(lane, i));
        out[i / 2] = add2(out[i / 2], pair(v.x, v.y));
        out[i / 2 + 1] = add2(out[i / 2 + 1], pair(v.z, v.w));
      }
      __syncwarp();
      if (first) mine[id] = 0.f;
    }
    if (sigmoid) {
      if (!dense) {
#pragma unroll
        for (int i = 0; i < NV; i += 2)
          away[i / 2] = pair(Sigmoid(now.value(i)).away(now.value(i)), Sigmoid(now.value(i + 1)).away(now.value(i + 1)));
      }
#pragma unroll
      for (int i = 0; i < NV / 2; ++i) out[i] = mul2(out[i], away[i]);
    }
    if (!there) continue;
    char* to = static_cast<char*>(a.dlogits[r]) + row * E * Elem<DT>::kBytes;
    constexpr int kPer = 16 / Elem<DT>::kBytes;
#pragma unroll
    for (int q = 0; q < NV / kPer; ++q) {
      const int c = gate_column<L>(lane, q * kPer);
      if (c >= E) continue;
      uint32_t o[4];
      pack2<DT, kPer / 2>(out + q * kPer / 2, o);
      if (vec) {
        store_raw<DT, kPer>(to, c, o);
      } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (c + i < E) store_one<DT>(to, c + i, o, i);
      }
    }
  }
}

}  // namespace

cudaError_t launch_gate_grad(int dt, bool gates, bool balance, GateArgs* args, cudaStream_t s) {
  size_t rows[kMoeMaxRanks];
  for (int r = 0; r < args->p; ++r) rows[r] = args->parts.rows[r];
  return by_row(dt, args->num_experts, gates ? args->k : 1, [&](auto d, auto lanes, auto nv) {
    constexpr int DT = decltype(d)::value, L = decltype(lanes)::value, NV = decltype(nv)::value;
    cut_rows(&args->parts, rows, args->p, 152 * 8, kThreads / L, false);
    return launch_gate_parts(!gates    ? gate_grad_kernel<DT, L, NV, false, true>
                             : balance ? gate_grad_kernel<DT, L, NV, true, true>
                                       : gate_grad_kernel<DT, L, NV, true, false>,
                             *args, kThreads, 0, s);
  });
}

}  // namespace ccl
