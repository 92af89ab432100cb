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
// Logits are read once and gradients written once; beside HBM, instructions bound
// it, some 270 a row of 256 with both parts.  Measured: 8 ranks x 16384 rows of 256 bf16,
// top-8 and the loss, 45 us (3.2 TB/s); the loss alone, fp32 and sigmoid, 46 us (5.8
// TB/s); 4 x 20001... rows of 60 fp32, top-6, 8.9 us.
#include "gate_rows.cuh"

namespace ccl {
namespace {

// A batch's choices are settled first, in all lanes; then every pass makes a row's
// gradients.  The next row, and the next batch's choices, are on the way meanwhile.
// Two CTAs a SM of 257 to 512 columns, but with both parts, which need more registers:
// the loss's gradient of 4 x 16384 rows of 384 fp32, sigmoid, takes 46 us so, 66 in one.
template <int DT, int L, int NV, int KM, bool GATES, bool BALANCE>
__global__ void __launch_bounds__(kThreads, NV == 8 ? 4 : NV == 16 && !(GATES && BALANCE) ? 2 : 1) gate_grad_kernel(const __grid_constant__ GateArgs a) {
  using Batch = GateBatch<L, KM>;
  constexpr int C = Batch::kChoices, kTeams = 32 / L, kWarps = kThreads / 32;
  // GATES: of each team, what the choices of its row add to their columns; zeros between rows
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
  float* mine = spread + (warp * kTeams + team) * (L * NV);
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
  const uint32_t choice_row = (threadIdx.x & 31) / C, choice = (threadIdx.x & 31) % C, team_row = team * Batch::kPasses;
  uint64_t row0 = part.lo + static_cast<uint64_t>(warp) * Batch::kRows;
  GateRow<DT, NV> next;
  next.template load<L>(a.logits[r], row0 + team_row, E, lane, row0 + team_row < part.hi, vec);
  int next_id = -1;
  float next_d = 0.f;
  const auto fetch_choice = [&](uint64_t row) {
    next_id = -1;
    next_d = 0.f;
    if (choice < k && row < part.hi) {
      next_id = a.ids_in[r][row * k + choice];
      next_d = a.dgates[r][row * k + choice];
    }
  };
  if constexpr (GATES) fetch_choice(row0 + choice_row);
  for (; row0 < part.hi; row0 += kWarps * Batch::kRows) {
    int id = next_id;
    float own = 0.f, value = -INFINITY, d = 0.f;  // own: what this lane's choice adds to its column
    bool first = false, twice = false;
    if constexpr (GATES) {
      const uint64_t row = row0 + choice_row;
      if (id < 0 || id >= E) id = -1;
      if (id >= 0) {
        d = a.scale * next_d;  // beside a choice that is none stands anything
        value = gate_logit<DT>(a.logits[r], row, E, id);
      }
      fetch_choice(row + kWarps * Batch::kRows);
      if (a.normalize) {
        // over the chosen ones' largest, which may be far below the row's
        const float base = base_of(lanes_max<C>(value), sigmoid), u = id >= 0 ? score_of(value, base, sigmoid) : 0.f;
        const float over = lanes_sum<C>(u), g = over == 0.f ? 0.f : quotient(u, over, reciprocal_of(over));
        const float mean = lanes_sum<C>(g * d);
        own = g * (d - mean);
      } else if (sigmoid) {
        own = id >= 0 ? sigmoid_score(value, 0.f) * d : 0.f;
      }
      // an expert that the token has twice is added up by the first lane of it
      bool again = false;
#pragma unroll
      for (int o = 1; o < C; ++o) again |= __shfl_xor_sync(kAllLanes, id, o) == id && (choice ^ o) < choice;
      first = id >= 0 && !again;
      twice = __any_sync(kAllLanes, id >= 0 && again);
    }
#pragma unroll 1
    for (int j = 0; j < Batch::kPasses; ++j) {
      const uint64_t row = row0 + team_row + j;
      const int slot = lane - j * C;  // 0 .. C - 1 in the lanes of this row's choices
      const bool here = slot >= 0 && slot < C, there = row < part.hi;
      const GateRow<DT, NV> now = next;
      {
        const uint64_t ahead = row0 + team_row + (j + 1 < Batch::kPasses ? j + 1 : kWarps * Batch::kRows);
        next.template load<L>(a.logits[r], ahead, E, lane, ahead < part.hi, vec);
      }
      F2 out[NV / 2], away[NV / 2];
      float all = 0.f;  // of the gates' part, taken off every column by its share
      if (dense) {
        float top = now.value(0);
#pragma unroll
        for (int i = 1; i < NV; ++i) top = larger(top, now.value(i));
        const float base = base_of(lanes_max<L>(top), sigmoid);
        const float part_total = scores_of<DT, NV, true, true>(now, base, sigmoid, out, away);
        // The mean of a_e over the shares: for softmax, whose lone score is 1, by a sum over the scores beside theirs
        F2 product = both(0.f);
        float total, mean = 0.f, inv;
        if (BALANCE && !sigmoid) {
          if constexpr (BALANCE) {
#pragma unroll
            for (int i = 0; i < NV / 2; ++i) product = fma2(out[i], weight[i], product);
          }
          const float2 sums = lanes_sum<L>(part_total, total2(product));
          total = sums.x;
          inv = total == 0.f ? 0.f : reciprocal_of(total);
          mean = sums.y * inv;
        } else {
          total = lanes_sum<L>(part_total);
          inv = total == 0.f ? 0.f : reciprocal_of(total);
        }
        if (GATES && !(a.normalize || sigmoid)) {
          float v = 0.f;
          if (here && id >= 0) v = own = softmax_score(value, base) * inv * d;
          all = lanes_sum<L>(v);
        }
        // shares; a lone one is 1 to the bit, so that it has no gradient
        if (sigmoid) {
#pragma unroll
          for (int i = 0; i < NV / 2; ++i) {
            out[i] = quotient(out[i], total, both(inv));
            if constexpr (BALANCE) product = fma2(out[i], weight[i], product);
          }
          if constexpr (BALANCE) mean = lanes_sum<L>(total2(product));
        } else {
#pragma unroll
          for (int i = 0; i < NV / 2; ++i) out[i] = mul2(out[i], both(inv));
        }
        const bool both_parts = GATES && BALANCE && !(a.normalize || sigmoid);
#pragma unroll
        for (int i = 0; i < NV / 2; ++i) {
          F2 f = both(-all);
          if constexpr (BALANCE) {
            // the loss's part first: of a lone share it is 0, and so is what is left
            f = add2(weight[i], both(-mean));
            if (both_parts) f = add2(f, both(-all));
          }
          out[i] = mul2(out[i], f);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NV / 2; ++i) out[i] = both(0.f);
      }
      if constexpr (GATES) {
        float v = own;
        if (twice) {
          v = 0.f;
          for (int q = 0; q < C; ++q) {
            const float more = __shfl_sync(kAllLanes, own, q, C);
            if (__shfl_sync(kAllLanes, id, q, C) == id) v += more;
          }
        }
        if (here && first) mine[id] = v;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NV; i += 4) {
          const float4 more = *reinterpret_cast<const float4*>(mine + gate_column<L>(lane, i));
          out[i / 2] = add2(out[i / 2], pair(more.x, more.y));
          out[i / 2 + 1] = add2(out[i / 2 + 1], pair(more.z, more.w));
        }
        __syncwarp();
        if (here && first) mine[id] = 0.f;
        __syncwarp();  // before the next row's
      }
      if (sigmoid) {
        if (!dense) {
#pragma unroll
          for (int i = 0; i < NV; i += 2) {  // NaN of a NaN, of which no base tells here
            const float x = now.value(i), y = now.value(i + 1), t = exp_of(-fabsf(x)), u = exp_of(-fabsf(y));
            away[i / 2] = pair(Sigmoid(t, rough_reciprocal(1.f + t)).away(x), Sigmoid(u, rough_reciprocal(1.f + u)).away(y));
          }
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
}

}  // namespace

cudaError_t launch_gate_grad(int dt, bool gates, bool balance, GateArgs* args, cudaStream_t s) {
  size_t rows[kMoeMaxRanks];
  for (int r = 0; r < args->p; ++r) rows[r] = args->parts.rows[r];
  return by_row(dt, args->num_experts, gates ? args->k : 1, [&](auto d, auto lanes, auto nv) {
    constexpr int DT = decltype(d)::value, L = decltype(lanes)::value, NV = decltype(nv)::value;
    const auto go = [&](auto km) {
      constexpr int KM = decltype(km)::value;
      // as many parts as are there at once: 8 x 16384 rows of 256 bf16 took 43 us so, 47 in twice as many, 53 in three quarters
      cut_rows(&args->parts, rows, args->p, 152 * 4, kThreads / 32 * GateBatch<L, KM>::kRows, false);
      auto* kernel = balance ? gate_grad_kernel<DT, L, NV, KM, true, true> : gate_grad_kernel<DT, L, NV, KM, true, false>;
      if constexpr (KM == 8) {
        if (!gates) kernel = gate_grad_kernel<DT, L, NV, KM, false, true>;
      }
      return launch_gate_parts(kernel, *args, kThreads, 0, s);
    };
    if constexpr (L >= 16) {
      if (gates && args->k > 8) return go(std::integral_constant<int, 16>{});
    }
    return go(std::integral_constant<int, 8>{});
  });
}

}  // namespace ccl
