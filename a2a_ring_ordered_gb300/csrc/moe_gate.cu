// moe_gate.cu -- the router's choice and its balance loss.
//
// A token's logits l, scores u (exp(l) or 1 / (1 + exp(-l))), shares p = u / sum u.
// The choice is the k largest logits; gates are u over the chosen ones' sum, or
// p, or u.  The loss is L = E / (k T^2) sum_e c_e sum_t p_te, c the counts.
//
// A row is read once; what bounds this is the instructions of the choice, some 300
// a row of 256 with top-8 and the loss, half of them on the ALU pipe, which is 74 %
// busy.  Measured: 8 ranks x 16384 rows of 256 bf16 with the loss 46 us (HBM would
// take 11), of one rank without it 34; 4 x 20001... rows of 60 fp32, top-6, 10 us; 8 rows
// 3.0 us in a captured graph.
#include <cooperative_groups.h>

#include <algorithm>

#include "gate_rows.cuh"

namespace ccl {
namespace {

__host__ __device__ constexpr int gate_threads(int nv) { return nv == 8 ? 512 : 256; }
constexpr size_t kCapSharedBytes = 80 * 1024;  // more than a third of a SM's, more than any row needs

// A column's place in the order of the choice: the logit's bits made to order as
// numbers do (-0 as 0, NaN above all), and under them 1023 - column, so that
// the larger key is the choice's next and keys are unlike.  bf16 fits whole, into
// the upper half; of fp32 the upper 22 bits do, and choices that these leave open
// are made again from all bits (1 % of rows of 256 normals, 40 % where they are bf16
// values: 8 x 16384 rows 47 and 82 us).  What is below kLeastKey is -inf, and no choice.
template <int DT>
__device__ constexpr uint32_t kLeastKey = DT == kF32 ? 0x2000u << 10 : 0x80u << 16;

__device__ __forceinline__ uint32_t ordered_bits(float l) {
  const uint32_t b = __float_as_uint(l + 0.0f);  // -0 becomes 0, a NaN the canonical one
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

template <int DT, int NV, int L>
__device__ __forceinline__ void make_keys(const GateRow<DT, NV>& row, int lane, uint32_t* key) {
  if constexpr (DT == kF32) {
#pragma unroll
    for (int i = 0; i < NV; ++i) key[i] = (ordered_bits(row.value(i)) & ~1023u) | static_cast<uint32_t>(1023 - gate_column<L>(lane, i));
  } else {
    const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; i += 2) {
      const __nv_bfloat162 v = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&row.w[i / 2]), zero);
      const uint32_t b = *reinterpret_cast<const uint32_t*>(&v);
      uint32_t signs;  // of both halves, in all of their bits
      asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(signs) : "r"(b));
      const uint32_t o = b ^ (signs | 0x80008000u);
      key[i] = o * 65536u + static_cast<uint32_t>(1023 - gate_column<L>(lane, i));
      key[i + 1] = (o & 0xFFFF0000u) | static_cast<uint32_t>(1023 - gate_column<L>(lane, i + 1));
    }
  }
}

__device__ __forceinline__ void order(uint32_t& a, uint32_t& b) {
  const uint32_t t = max(a, b);
  b = min(a, b);
  a = t;
}
// Eight keys, largest first: Batcher's odd-even merge sort.
__device__ __forceinline__ void sort8(uint32_t* x) {
  order(x[0], x[1]), order(x[2], x[3]), order(x[4], x[5]), order(x[6], x[7]);
  order(x[0], x[2]), order(x[1], x[3]), order(x[4], x[6]), order(x[5], x[7]);
  order(x[1], x[2]), order(x[5], x[6]);
  order(x[0], x[4]), order(x[1], x[5]), order(x[2], x[6]), order(x[3], x[7]);
  order(x[2], x[4]), order(x[3], x[5]);
  order(x[1], x[2]), order(x[3], x[4]), order(x[5], x[6]);
}

// The keys of the k choices, largest first, to `into` (of the team; by the lane whose
// each is); the largest key.  `open`: the keys do not tell the choices apart, or the
// last of them from the next.  FULL: k is KM.
template <int DT, int NV, int L, int KM, bool FULL>
__device__ __forceinline__ uint32_t choose(uint32_t* key, int k, uint32_t* into, bool& open) {
  uint32_t top = 0, last = 0;
  open = false;
  if constexpr (NV == 8) sort8(key);
#pragma unroll
  for (int j = 0; j < KM + (DT == kF32 ? 1 : 0); ++j) {
    if (!FULL && (j > k || (DT != kF32 && j == k))) break;
    uint32_t head = key[0];
    if constexpr (NV != 8) {
      // what is left is below the last choice, in every lane
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        key[i] = j == 0 || key[i] < last ? key[i] : 0;
        head = i == 0 ? key[0] : max(head, key[i]);
      }
    }
    const uint32_t most = lanes_max<L>(head);
    if constexpr (DT == kF32) open |= j > 0 && (most ^ last) < 1024 && most >= kLeastKey<DT>;
    if (j == 0) top = most;
    last = most;
    if (head == most) {
      if (j < KM && (FULL || DT != kF32 || j < k)) into[j] = most;
      if constexpr (NV == 8) {
        // no more than the choices that are left can come from here
        constexpr int kLeft = KM + (DT == kF32 ? 1 : 0) - 1;
#pragma unroll
        for (int i = 0; i < 7; ++i)
          if (i < kLeft - j) key[i] = key[i + 1];
        if (7 < KM + 1 - j) key[7] = 0;
      }
    }
  }
  return top;
}

// Choice number `slot` from all 32 bits of each logit, or -1.
template <int NV, int L>
__device__ __forceinline__ int choose_exactly(const GateRow<kF32, NV>& row, int lane, int slot, int k) {
  uint32_t bits[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) bits[i] = row.value(i) == -INFINITY ? 0 : ordered_bits(row.value(i));
  int mine = -1;
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0, at = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (bits[i] > best) {
        best = bits[i];
        at = gate_column<L>(lane, i);
      }
    const uint32_t most = lanes_max<L>(best);
    const uint32_t first = lanes_min<L>(best == most ? at : 0x7FFFFFFF);
    if (slot == j && most != 0) mine = static_cast<int>(first);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (gate_column<L>(lane, i) == static_cast<int>(first)) bits[i] = 0;
  }
  return mine;
}

__device__ __forceinline__ float bf16_of_key(uint32_t key) {
  const uint32_t o = key >> 16;
  return __uint_as_float((o & 0x8000u ? o ^ 0x8000u : ~o) << 16);
}

// Every pass chooses in a row and adds its shares; the batch's gates follow, in all
// lanes.  The next row is on the way meanwhile.
template <int DT, int L, int NV, int KM, bool SELECT, bool BALANCE>
__global__ void __launch_bounds__(gate_threads(NV)) gate_kernel(const __grid_constant__ GateArgs a) {
  using Batch = GateBatch<L, KM>;
  constexpr int C = Batch::kChoices, kTeams = 32 / L, kWarps = gate_threads(NV) / 32;
  extern __shared__ float shared[];  // BALANCE: [kWarps][kTeams][L * NV] sums of shares, then E + 1 counts
  __shared__ uint32_t chosen_keys[SELECT ? kWarps : 1][32];  // of a warp's batch, where its lanes look for their choices
  pdl_enter();
  const int lane = threadIdx.x & (L - 1), warp = threadIdx.x >> 5, team = (threadIdx.x & 31) / L, E = a.num_experts, k = a.k;
  const bool sigmoid = a.score == CCL_SCORE_SIGMOID, vec = a.vec != 0;
  const bool dense = BALANCE || !(a.normalize || sigmoid);  // whether shares, over all of a row, are wanted
  const RowPart part = row_part(a.parts, a.p, blockIdx.x);
  const int r = part.r;
  int* counts = reinterpret_cast<int*>(shared + kWarps * kTeams * L * NV);
  F2 sums[NV / 2];
  int live_rows = 0;
  if constexpr (BALANCE) {
#pragma unroll
    for (int i = 0; i < NV / 2; ++i) sums[i] = both(0.f);
    for (int i = threadIdx.x; i <= E; i += gate_threads(NV)) counts[i] = 0;
    __syncthreads();
  }
  // rows of the batch that this lane's choice, and this team's pass 0, are in
  const uint32_t choice_row = (threadIdx.x & 31) / C, team_row = team * Batch::kPasses;
  uint64_t row0 = part.lo + static_cast<uint64_t>(warp) * Batch::kRows;
  GateRow<DT, NV> next;
  next.template load<L>(a.logits[r], row0 + team_row, E, lane, row0 + team_row < part.hi, vec);
  for (; row0 < part.hi; row0 += kWarps * Batch::kRows) {
    int id = -1;
    float value = -INFINITY, base = 0.f, total = 0.f;  // of this lane's choice and its row
#pragma unroll 1
    for (int j = 0; j < Batch::kPasses; ++j) {
      const int slot = lane - j * C;  // 0 .. C - 1 in the lanes of this row's choices
      const GateRow<DT, NV> now = next;
      {
        const uint64_t ahead = row0 + team_row + (j + 1 < Batch::kPasses ? j + 1 : kWarps * Batch::kRows);
        next.template load<L>(a.logits[r], ahead, E, lane, ahead < part.hi, vec);
      }
      float top = -INFINITY;
      if constexpr (SELECT) {
        uint32_t key[NV];
        bool open;
        make_keys<DT, NV, L>(now, lane, key);
        uint32_t* const into = chosen_keys[warp] + (threadIdx.x & 31) - lane + j * C;
        const uint32_t top_key = k == KM ? choose<DT, NV, L, KM, true>(key, k, into, open) : choose<DT, NV, L, KM, false>(key, k, into, open);
        if constexpr (DT == kF32) {
          __syncwarp();
          // by column, as the other way to choose gives them
          int column = -1;
          const bool mine = slot >= 0 && slot < k;
          if (mine && into[slot] >= kLeastKey<DT>) column = 1023 - static_cast<int>(into[slot] & 1023u);
          if (__any_sync(kAllLanes, open)) column = choose_exactly<NV, L>(now, lane, slot, k);
          if (mine) id = column;
        } else {
          top = top_key >= kLeastKey<DT> ? bf16_of_key(top_key) : -INFINITY;
        }
        live_rows += top_key >= kLeastKey<DT>;  // counted in lane 0
      }
      if (dense) {
        if constexpr (!SELECT || DT == kF32) {
          top = now.value(0);
#pragma unroll
          for (int i = 1; i < NV; ++i) top = larger(top, now.value(i));
          top = lanes_max<L>(top);
        }
        const float row_base = base_of(top, sigmoid);
        F2 u[NV / 2];
        const float row_total = lanes_sum<L>(scores_of<DT, NV, !SELECT, false>(now, row_base, sigmoid, u, nullptr));
        if (SELECT && slot >= 0 && slot < C) {
          base = row_base;
          total = row_total;
        }
        if constexpr (BALANCE) {
          const F2 inv = both(row_total == 0.f ? 0.f : rough_reciprocal(row_total));
#pragma unroll
          for (int i = 0; i < NV / 2; ++i) sums[i] = fma2(u[i], inv, sums[i]);
        }
      }
      if constexpr (!SELECT) {
        bool live = false;
#pragma unroll
        for (int i = 0; i < NV; ++i) live |= !(now.value(i) == -INFINITY);
        live_rows += (__ballot_sync(kAllLanes, live) >> (team * L) & static_cast<unsigned>((1ull << L) - 1)) != 0;
      }
    }
    const int choice = (threadIdx.x & 31) % C;
    const uint64_t row = row0 + choice_row, item = row * k + choice;
    const bool there = row < part.hi && choice < k;
    if constexpr (SELECT) {
      if constexpr (DT == kF32) {
        if (id >= 0) value = gate_logit<DT>(a.logits[r], row, E, id);
      } else {
        __syncwarp();
        const uint32_t key = chosen_keys[warp][threadIdx.x & 31];
        if (choice < k && key >= kLeastKey<DT>) {
          id = 1023 - static_cast<int>(key & 1023u);
          value = bf16_of_key(key);
        }
      }
      __syncwarp();  // before the next batch's keys
      float g = 0.f;
      if (a.normalize) {
        const float own_base = base_of(__shfl_sync(kAllLanes, value, 0, C), sigmoid), own = id >= 0 ? score_of(value, own_base, sigmoid) : 0.f;
        const float over = lanes_sum<C>(own);
        if (id >= 0) g = over == 0.f ? 0.f : quotient(own, over, reciprocal_of(over));
      } else if (id >= 0) {
        g = sigmoid ? sigmoid_score(value, 0.f) : quotient(softmax_score(value, base), total, reciprocal_of(total));
      }
      if (there) {
        a.ids[r][item] = id;
        a.gates[r][item] = a.scale * g;
      }
    } else {
      if (there) id = a.ids_in[r][item];
      if (id >= E) id = -1;
    }
    if constexpr (BALANCE)
      if (id >= 0) atomicAdd(counts + id, 1);
  }
  if constexpr (BALANCE) {
#pragma unroll
    for (int i = 0; i < NV; i += 2)
      *reinterpret_cast<float2*>(shared + (warp * kTeams + team) * (L * NV) + gate_column<L>(lane, i)) = parts(sums[i / 2]);
    if (lane == 0) atomicAdd(counts + E, live_rows);
    __syncthreads();
    float* out = a.partial + blockIdx.x * balance_part_words(E);
    for (int e = threadIdx.x; e <= E; e += gate_threads(NV)) {
      if (e < E) {
        float s = 0.f;
        for (int w = 0; w < kWarps * kTeams; ++w) s += shared[w * (L * NV) + e];
        out[e] = s;
      }
      reinterpret_cast<int*>(out)[E + e] = counts[e];
    }
  }
}

// A cluster of CTAs per rank adds up the parts of its own, or of all where the
// ranks' tokens are one batch.  A CTA has 32 experts at a time, each of its warps
// every 32nd part; then a warp has an expert, adds up what the warps have of it
// and multiplies by its count; the cluster's first CTA adds up the products.  The
// roundings of all of that are kept beside the sums (Knuth's two-sum, products by
// a fused multiply-add): additions of 64 bits take 16 times as long here as two of
// those.
constexpr int kJoinThreads = 1024, kJoinWarps = kJoinThreads / 32, kJoinCluster = 8;
struct Kept {
  float sum = 0.f, rest = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float t = sum + v, back = t - sum;
    rest += (sum - (t - back)) + (v - back);
    sum = t;
  }
  __device__ __forceinline__ void add(const Kept& o) {
    add(o.sum);
    rest += o.rest;
  }
  __device__ __forceinline__ void add_lanes() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      Kept other;
      other.sum = __shfl_xor_sync(kAllLanes, sum, o);
      other.rest = __shfl_xor_sync(kAllLanes, rest, o);
      add(other);
    }
  }
};
__global__ void __launch_bounds__(kJoinThreads) balance_join_kernel(const __grid_constant__ BalanceJoinArgs a) {
  namespace cg = cooperative_groups;
  __shared__ float sums[kJoinWarps][33], rests[kJoinWarps][33];
  __shared__ int numbers[kJoinWarps][33], warp_rows[kJoinWarps];
  __shared__ float warp_sums[kJoinWarps][2];
  __shared__ float cta_sum[2];
  pdl_enter();
  cg::cluster_group cluster = cg::this_cluster();
  const int r = blockIdx.y, E = a.num_experts, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = static_cast<int>(cluster.block_rank()), ctas = static_cast<int>(cluster.num_blocks());
  const uint32_t lo = a.together ? 0 : a.first[r], hi = a.together ? a.first[a.p] : a.first[r + 1];
  const size_t words = balance_part_words(E);
  Kept product;  // of the warp's experts, in all lanes
  for (int e0 = c0 * 32; e0 < E; e0 += ctas * 32) {
    Kept s;
    int c = 0;
    if (e0 + lane < E) {
      const float* at = a.partial + (lo + warp) * words + e0 + lane;
#pragma unroll 4
      for (uint32_t i = lo + warp; i < hi; i += kJoinWarps, at += kJoinWarps * words) {
        s.add(at[0]);
        c += reinterpret_cast<const int*>(at)[E];
      }
    }
    sums[warp][lane] = s.sum;
    rests[warp][lane] = s.rest;
    numbers[warp][lane] = c;
    __syncthreads();
    s.sum = sums[lane][warp];
    s.rest = rests[lane][warp];
    s.add_lanes();
    c = __reduce_add_sync(kAllLanes, numbers[lane][warp]);
    __syncthreads();
    if (e0 + warp >= E) continue;
    if (lane == 0) a.counts[r][e0 + warp] = c;
    // the count in two numbers that are exact
    const float high = static_cast<float>(c & ~4095), low = static_cast<float>(c & 4095);
    Kept p;
    p.sum = s.sum * high;
    p.rest = fmaf(s.sum, high, -p.sum) + s.rest * static_cast<float>(c);
    const float more = s.sum * low;
    p.rest += fmaf(s.sum, low, -more);
    p.add(more);
    product.add(p);
  }
  int rows = 0;
  if (c0 == 0) {
    for (uint32_t i = lo + threadIdx.x; i < hi; i += kJoinThreads) rows += reinterpret_cast<const int*>(a.partial)[i * words + 2 * E];
    rows = __reduce_add_sync(kAllLanes, rows);
  }
  if (lane == 0) {
    warp_sums[warp][0] = product.sum;
    warp_sums[warp][1] = product.rest;
    warp_rows[warp] = rows;
  }
  __syncthreads();
  if (warp == 0) {
    product.sum = warp_sums[lane][0];
    product.rest = warp_sums[lane][1];
    product.add_lanes();
    rows = __reduce_add_sync(kAllLanes, warp_rows[lane]);
    if (lane == 0) {
      cta_sum[0] = product.sum;
      cta_sum[1] = product.rest;
    }
  }
  cluster.sync();
  if (c0 == 0 && threadIdx.x == 0) {
    for (int q = 1; q < ctas; ++q) {
      const float* other = cluster.map_shared_rank(cta_sum, q);
      Kept p;
      p.sum = other[0];
      p.rest = other[1];
      product.add(p);
    }
    a.counts[r][E] = rows;
    const float t = static_cast<float>(rows);
    a.losses[r][0] = rows == 0 ? 0.f : (product.sum + product.rest) / t * (static_cast<float>(E) / a.k) / t;
  }
  cluster.sync();  // the first CTA has read the others' sums
}

}  // namespace

cudaError_t launch_gate(int dt, bool select, bool balance, GateArgs* args, cudaStream_t s) {
  size_t rows[kMoeMaxRanks];
  for (int r = 0; r < args->p; ++r) rows[r] = args->parts.rows[r];
  return by_row(dt, args->num_experts, args->k, [&](auto d, auto lanes, auto nv) {
    constexpr int DT = decltype(d)::value, L = decltype(lanes)::value, NV = decltype(nv)::value, kWarps = gate_threads(NV) / 32;
    size_t smem = balance ? (static_cast<size_t>(kWarps) * 32 * NV + args->num_experts + 1) * 4 : 0;
    const auto go = [&](auto km) {
      constexpr int KM = decltype(km)::value;
      // a batch a warp at least, then parts for two CTAs a SM: six without the loss, where they would fit, took 12.1 us for 61,998 rows of 60
      // fp32 instead of 9.8
      cut_rows(&args->parts, rows, args->p, kBalanceParts, kWarps * GateBatch<L, KM>::kRows, balance);
      auto* kernel = !select ? gate_kernel<DT, L, NV, KM, false, true> : balance ? gate_kernel<DT, L, NV, KM, true, true> : gate_kernel<DT, L, NV, KM, true, false>;
      // no third CTA on a SM, where registers would let one on: the parts are two a SM, and while the call before still has some SMs
      // it would be missing from another.  The loss of given ids of 4 x 16384 rows of 384 bf16, call after call, 32 us -> 26
      if (NV == 16 && !select) {
        smem = kCapSharedBytes;
        const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (err != cudaSuccess) return err;
      }
      return launch_gate_parts(kernel, *args, gate_threads(NV), smem, s);
    };
    if constexpr (L >= 16) {
      if (args->k > 8) return go(std::integral_constant<int, 16>{});
    }
    return go(std::integral_constant<int, 8>{});
  });
}

cudaError_t launch_balance_join(const BalanceJoinArgs& a, cudaStream_t s) {
  const int ctas = std::min((a.num_experts + 31) / 32, kJoinCluster);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(a.p));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = CCL_PDL ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, balance_join_kernel, a);
  if (err == cudaSuccess) note_launch();
  return err;
}

}  // namespace ccl
