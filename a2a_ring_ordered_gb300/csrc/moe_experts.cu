// moe_experts.cu -- a rank's tokens in the order of its experts, and back.
//
// Row of (token t, choice j), with e its expert among the rank's own:
//   row(t, j) = #{(t', j') of an expert before e}
//             + #{(t', j') before (t, j) in token-choice order, of expert e},
// a stable counting sort.  Then sorted[row(t, j)] = x[t] (to_experts),
// out[t] = sum_j w[t][j] y[row(t, j)] (from_experts), and the gradient of the
// latter, dy[row(t, j)] = w[t][j] dout[t], dw[t][j] = <y[row(t, j)], dout[t]>.
// The sort is bound by latency, the others move rows and are bound by HBM.
// Measured, 8 choices of 256 experts, rows of 7168 bf16: the sort of 4096 items
// 3.3 us, of 1,048,576 77 us; 8 ranks x 2048 tokens: sort and to_experts 324 us
// (6.5 TB/s), the gradient 614 us (6.5 TB/s); 8 ranks x 4096: from_experts 636
// us (6.65 TB/s).
#include <cooperative_groups.h>

#include "device_common.cuh"
#include "realign.cuh"

namespace ccl {
namespace {

constexpr int kSortMaxCluster = 16;
constexpr uint32_t kSortMaxWarps = 32;
constexpr int kSortUnroll = 4;           // id loads in flight per lane
constexpr uint32_t kPerTurn = 32 * kSortUnroll;  // items that a warp takes at a time
constexpr unsigned kAll = 0xFFFFFFFFu;

// The expert of an item among the rank's own, or -1.
__device__ __forceinline__ int sort_expert(const int32_t* ids, uint32_t i, uint32_t hi, int first, int experts) {
  if (i >= hi) return -1;
  const int64_t e = static_cast<int64_t>(ids[i]) - first;
  return (e >= 0 && e < experts) ? static_cast<int>(e) : -1;
}

// kSortUnroll groups of 32 items of one warp: each lane's experts, and the lanes
// that hold the same one (with the same low `bits` bits), by one vote per bit.
struct SortItems {
  int e[kSortUnroll];
  unsigned same[kSortUnroll];
  __device__ __forceinline__ SortItems(const int32_t* ids, uint32_t b, uint32_t hi, int first, int experts, int bits) {
    const uint32_t lane = threadIdx.x & 31;
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u) {
      e[u] = sort_expert(ids, b + 32 * u + lane, hi, first, experts);
      same[u] = kAll;
    }
    for (int i = 31; i > 31 - bits; --i)
#pragma unroll
      for (int u = 0; u < kSortUnroll; ++u) {
        const int one = e[u] << i >> 31;  // the bit, in all places
        same[u] &= ~(__ballot_sync(kAll, one < 0) ^ static_cast<unsigned>(one));
      }
  }
};

// One cluster of CTAs per rank (grid x = CTA in the cluster, grid y = rank).
// CTA c owns a contiguous range of the rank's items and warp w of it a
// contiguous part of that, so walking parts in order keeps the sort stable.
//  1. Each warp counts its part's items per expert in its own row of
//     hist (the first of the lanes of one expert adds the group), so nothing
//     is atomic.
//  2. A column of hist becomes the running count of the warps before; the
//     CTAs' totals are exchanged through distributed shared memory; a scan
//     over the experts gives every expert its first row.
//  3. The warp walks its part again (its first turn's items are still in
//     registers: most parts are no longer): row = hist entry + rank among the
//     lanes of the same expert, and the entry moves on by the group.
__global__ void moe_sort_kernel(const __grid_constant__ MoeSortArgs a) {
  namespace cg = cooperative_groups;
  extern __shared__ uint32_t smem[];
  const int E = a.num_experts;
  const int bits = 33 - __clz(E);  // they tell 0 .. E - 1 and -1 apart, with one to spare
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  uint32_t* hist = smem;             // [warps][E]
  uint32_t* total = hist + warps * E;  // [E]: this CTA's items of each expert
  uint32_t* base = total + E;          // [E]: first row of the CTA's items of each expert
  __shared__ uint32_t warp_sum[32];
  cg::cluster_group cluster = cg::this_cluster();
  const uint32_t c = cluster.block_rank(), ctas = cluster.num_blocks();
  const int r = blockIdx.y;
  for (int i = tid; i < warps * E; i += blockDim.x) hist[i] = 0;
  pdl_enter();
  const int32_t* ids = a.ids[r];
  const int first = a.first[r];
  const uint32_t items = a.items[r];
  // items per warp: whole groups of 32 lanes
  const uint32_t parts = ctas * warps;
  const uint32_t part = ((items + parts - 1) / parts + 31) / 32 * 32;
  const uint64_t lo64 = static_cast<uint64_t>(c * warps + warp) * part;
  const uint32_t lo = lo64 < items ? static_cast<uint32_t>(lo64) : items;
  const uint32_t hi = items - lo < part ? items : lo + part;
  uint32_t* mine = hist + warp * E;
  __syncthreads();

  const auto count = [&](const SortItems& x) {
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u) {
      if (x.e[u] >= 0 && lane == __ffs(x.same[u]) - 1) mine[x.e[u]] += __popc(x.same[u]);
      __syncwarp();
    }
  };
  const SortItems held(ids, lo, hi, first, E, bits);  // all that most warps have
  count(held);
  for (uint32_t b = lo + kPerTurn; b < hi; b += kPerTurn) count(SortItems(ids, b, hi, first, E, bits));
  __syncthreads();
  for (int e = tid; e < E; e += blockDim.x) {
    uint32_t run = 0;
    for (int w0 = 0; w0 < warps; w0 += 8) {  // warps is a multiple of 8
      uint32_t v[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) v[w] = hist[(w0 + w) * E + e];
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        hist[(w0 + w) * E + e] = run;
        run += v[w];
      }
    }
    total[e] = run;
  }
  cluster.sync();
  // experts in blocks of blockDim.x: this thread's expert, its rows in all
  // CTAs and in the CTAs before this one, then a scan over the threads
  uint32_t carry = 0;
  for (int e0 = 0; e0 < E; e0 += blockDim.x) {
    const int e = e0 + tid;
    uint32_t all = 0, before = 0;
    if (e < E) {
      for (uint32_t q = 0; q < ctas; ++q) {
        const uint32_t v = cluster.map_shared_rank(total, q)[e];
        all += v;
        before += q < c ? v : 0;
      }
    }
    uint32_t incl = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += t;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    uint32_t start = carry, round = 0;
    for (int w = 0; w < warps; ++w) {
      const uint32_t v = warp_sum[w];
      start += w < warp ? v : 0;
      round += v;
    }
    start += incl - all;
    carry += round;
    if (e < E) {
      base[e] = start + before;
      if (c == 0) a.offsets[r][e] = static_cast<int32_t>(start);
    }
    __syncthreads();
  }
  if (c == 0 && tid == 0) a.offsets[r][E] = static_cast<int32_t>(carry);
  cluster.barrier_arrive();  // the other CTAs may still read this one's totals

  int32_t* rows = a.rows[r];
  const auto place = [&](const SortItems& x, uint32_t b) {
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u) {
      const uint32_t i = b + 32 * u + lane;
      const uint32_t before = __popc(x.same[u] & ((1u << lane) - 1u));
      const uint32_t at = x.e[u] >= 0 ? mine[x.e[u]] : 0;
      __syncwarp();
      if (x.e[u] >= 0 && before == 0) mine[x.e[u]] = at + __popc(x.same[u]);
      __syncwarp();
      if (i < hi) rows[i] = x.e[u] >= 0 ? static_cast<int32_t>(base[x.e[u]] + at + before) : -1;
    }
  };
  place(held, lo);
  for (uint32_t b = lo + kPerTurn; b < hi; b += kPerTurn) place(SortItems(ids, b, hi, first, E, bits), b);
  cluster.barrier_wait();
}

// ------------------------------------------------------------------ rows
// f / n and f % n; a 32-bit division wherever it serves.
struct Split {
  uint64_t q;
  uint32_t r;
};
__device__ __forceinline__ Split split(uint64_t f, uint32_t n) {
  Split s;
  if ((f >> 32) == 0) {
    s.q = static_cast<uint32_t>(f) / n;
    s.r = static_cast<uint32_t>(f) - static_cast<uint32_t>(s.q) * n;
  } else {
    s.q = f / n;
    s.r = static_cast<uint32_t>(f - s.q * n);
  }
  return s;
}

// The row of a choice, or -1 where it has none in the buffer.
__device__ __forceinline__ int64_t row_of(const int32_t* rows, uint64_t item, uint32_t cap) {
  const int32_t row = __ldg(rows + item);
  return (row >= 0 && static_cast<uint32_t>(row) < cap) ? row : -1;
}

// A rank's (token, vector) pairs are one flat range (grid y = rank); each
// vector is read once and written to the token's k rows.
constexpr int kCopyVectors = 4;  // per thread, loaded together
__global__ void __launch_bounds__(kThreads) moe_to_experts_kernel(const __grid_constant__ MoeRowsArgs a, uint32_t nv) {
  constexpr int U = kCopyVectors;
  pdl_enter();
  const int r = blockIdx.y, k = a.k;
  const uint64_t total = static_cast<uint64_t>(a.tokens[r]) * nv;
  const uint64_t row_bytes = static_cast<uint64_t>(nv) * 16;
  const uint64_t f0 = (static_cast<uint64_t>(blockIdx.x) * U) * kThreads + threadIdx.x;
  if (f0 >= total) return;
  const char* x = static_cast<const char*>(a.x[r]);
  uint4 w[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (f0 + u * kThreads < total) w[u] = ld_once16(x + (f0 + u * kThreads) * 16);
  char* out = static_cast<char*>(a.out[r]);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint64_t f = f0 + u * kThreads;
    if (f >= total) continue;
    const Split at = split(f, nv);
    const uint64_t t = at.q, v = at.r;
    for (int j = 0; j < k; ++j) {
      const int64_t row = row_of(a.rows[r], t * k + j, a.cap[r]);
      if (row >= 0) st_stream16(out + row * row_bytes + v * 16, w[u]);
    }
  }
}

// ------------------------------------------------------------ off the grid
// Rows that do not all start on 16 bytes (odd widths, views): the written row
// is walked in its own aligned granules.  A whole granule is stored at once,
// from source bytes that two aligned loads hold, whatever their phase; the
// granules that the row shares with its neighbours, its first and its last,
// go element by element.
struct Granule {
  char* at;         // aligned
  uint32_t lo, hi;  // the row's bytes in it; none where lo == hi
  __device__ __forceinline__ bool any() const { return lo < hi; }
  __device__ __forceinline__ bool whole() const { return hi - lo == 16; }
};
__device__ __forceinline__ Granule granule_of(char* row, uint64_t row_bytes, uint64_t u) {
  const uintptr_t first = reinterpret_cast<uintptr_t>(row), end = first + row_bytes;
  const uintptr_t at = (first & ~static_cast<uintptr_t>(15)) + 16 * u;
  Granule g;
  g.at = reinterpret_cast<char*>(at);
  g.lo = at < first ? static_cast<uint32_t>(first - at) : 0u;
  g.hi = at >= end ? g.lo : at + 16 > end ? static_cast<uint32_t>(end - at) : 16u;
  return g;
}
// Stores the row's bytes of a granule.
template <int B>
__device__ __forceinline__ void store_granule(const Granule& g, const uint4 v) {
  if (g.whole()) {
    st_stream16(g.at, v);
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 16 / B; ++e) {
    const uint32_t at = e * B;
    if (at < g.lo || at >= g.hi) continue;
    if constexpr (B == 4) st_stream4(g.at + at, w[e]);
    else st_stream2(g.at + at, (e & 1) ? w[e / 2] >> 16 : w[e / 2] & 0xFFFFu);
  }
}
// Zeros in place of the bytes that are not the row's.
template <int B>
__device__ __forceinline__ uint4 only_row(const Granule& g, const uint4 v) {
  if (g.whole()) return v;
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 16 / B; ++e) {
    const uint32_t at = e * B;
    if (at >= g.lo && at < g.hi) continue;
    w[at / 4] &= B == 4 ? 0u : (e & 1) ? 0xFFFFu : 0xFFFF0000u;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Granules that a row of so many bytes can touch.
__host__ __device__ constexpr uint64_t granules(uint64_t row_bytes) { return (row_bytes + 30) / 16; }

// One flat range of (token, choice, granule of the choice's row) per rank,
// kOffUnits of them per thread with their loads on the way together.
constexpr int kOffUnits = 2;
template <int B>
__global__ void __launch_bounds__(kThreads) moe_to_experts_off_kernel(const __grid_constant__ MoeRowsArgs a, uint64_t row_bytes) {
  constexpr int U = kOffUnits;
  pdl_enter();
  const int r = blockIdx.y;
  const uint32_t ng = static_cast<uint32_t>(granules(row_bytes));
  const uint64_t items = static_cast<uint64_t>(a.tokens[r]) * a.k;
  const uint64_t f0 = static_cast<uint64_t>(blockIdx.x) * U * kThreads + threadIdx.x;
  Granule g[U];
  const char* from[U];
  uint4 w[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Split at = split(f0 + u * kThreads, ng);
    const int64_t row = at.q < items ? row_of(a.rows[r], at.q, a.cap[r]) : -1;
    char* to = static_cast<char*>(a.out[r]) + row * row_bytes;
    g[u].at = to;
    g[u].lo = g[u].hi = 0;
    if (row >= 0) g[u] = granule_of(to, row_bytes, at.r);
    // of the granule's first byte
    from[u] = static_cast<const char*>(a.x[r]) + static_cast<uint32_t>(at.q) / static_cast<uint32_t>(a.k) * row_bytes + (g[u].at - to);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) w[u] = load16_part(from[u], g[u].lo, g[u].hi);
#pragma unroll
  for (int u = 0; u < U; ++u) store_granule<B>(g[u], w[u]);
}

// One flat range of (token, granule of its output row) per rank; the rows of
// KB choices (all of them, or 8 at a time) are looked up together, then loaded
// together, before any is added.
template <int DT, int KB>
__global__ void __launch_bounds__(kThreads) moe_from_experts_off_kernel(const __grid_constant__ MoeRowsArgs a, uint64_t row_bytes) {
  constexpr int B = Elem<DT>::kBytes, N = 16 / B;
  pdl_enter();
  const int r = blockIdx.y, k = a.k;
  const Split at = split(static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x, static_cast<uint32_t>(granules(row_bytes)));
  const uint64_t t = at.q;
  if (t >= a.tokens[r]) return;
  char* to = static_cast<char*>(a.out[r]) + t * row_bytes;
  const Granule g = granule_of(to, row_bytes, at.r);
  if (!g.any()) return;
  const char* y = static_cast<const char*>(a.y[r]) + (g.at - to);  // of the granule's first byte, in row 0
  const float* weights = a.weights[r];
  float acc[N];
#pragma unroll
  for (int e = 0; e < N; ++e) acc[e] = -0.0f;  // -0 + x is x, to the bit
  bool have = false;
  for (int j0 = 0; j0 < k; j0 += KB) {
    uint4 raw[KB];
    int64_t row[KB];
    float wt[KB];
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      row[b] = j0 + b < k ? row_of(a.rows[r], t * k + j0 + b, a.cap[r]) : -1;
      wt[b] = (weights != nullptr && j0 + b < k) ? __ldg(weights + t * k + j0 + b) : 1.0f;
    }
#pragma unroll
    for (int b = 0; b < KB; ++b) raw[b] = load16_part(y + row[b] * static_cast<int64_t>(row_bytes), g.lo, row[b] >= 0 ? g.hi : g.lo);
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      if (row[b] < 0) continue;
      const uint32_t w[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
#pragma unroll
      for (int e = 0; e < N; ++e) acc[e] = __fadd_rn(acc[e], __fmul_rn(wt[b], widen<DT>(w, e)));
      have = true;
    }
  }
  if (!have) {
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.0f;
  }
  uint32_t w[4];
  pack_out<DT, N>(acc, w);
  store_granule<B>(g, make_uint4(w[0], w[1], w[2], w[3]));
}

// `tpi` lanes (a power of two, up to a warp) per (token, choice): its row is
// walked in the granules of dy's row (y's where only the gates are wanted), and
// the lanes' dot products are added in a fixed tree.
template <int DT>
__global__ void __launch_bounds__(kThreads) moe_from_experts_grad_off_kernel(const __grid_constant__ MoeRowsArgs a,
                                                                            uint64_t row_bytes, int tpi) {
  constexpr int B = Elem<DT>::kBytes, N = 16 / B, U = 2;
  pdl_enter();
  const int r = blockIdx.y;
  const uint32_t slot = threadIdx.x / tpi, in = threadIdx.x - slot * tpi;
  const uint64_t item = static_cast<uint64_t>(blockIdx.x) * (kThreads / tpi) + slot;
  const bool live = item < static_cast<uint64_t>(a.tokens[r]) * a.k;
  const int64_t row = live ? row_of(a.rows[r], item, a.cap[r]) : -1;
  const float wt = (live && a.weights[r] != nullptr) ? __ldg(a.weights[r] + item) : 1.0f;
  const uint64_t t = live ? static_cast<uint32_t>(item) / static_cast<uint32_t>(a.k) : 0;
  const char* dout = static_cast<const char*>(a.x[r]) + t * row_bytes;
  char* dy = static_cast<char*>(a.out[r]);
  float* dw = a.dweights[r];
  float dot = 0.0f;
  if (row >= 0) {
    const char* y = static_cast<const char*>(a.y[r]) + row * row_bytes;
    char* walked = dy != nullptr ? dy + row * row_bytes : const_cast<char*>(y);
    const uint32_t ng = static_cast<uint32_t>(granules(row_bytes));
    for (uint32_t u0 = in; u0 < ng; u0 += tpi * U) {
      Granule g[U];
      uint4 d[U], v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        g[u] = granule_of(walked, row_bytes, u0 + u * tpi);
        const int64_t into = g[u].at - walked;
        d[u] = load16_part(dout + into, g[u].lo, g[u].hi);
        v[u] = load16_part(y + into, g[u].lo, dw != nullptr ? g[u].hi : g[u].lo);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!g[u].any()) continue;
        const uint4 dc = only_row<B>(g[u], d[u]), vc = only_row<B>(g[u], v[u]);
        const uint32_t dq[4] = {dc.x, dc.y, dc.z, dc.w}, vq[4] = {vc.x, vc.y, vc.z, vc.w};
        float o[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float de = widen<DT>(dq, e);
          o[e] = __fmul_rn(wt, de);
          if (dw != nullptr) dot = fmaf(widen<DT>(vq, e), de, dot);
        }
        if (dy == nullptr) continue;
        uint32_t w[4];
        pack_out<DT, N>(o, w);
        store_granule<B>(g[u], make_uint4(w[0], w[1], w[2], w[3]));
      }
    }
  }
  for (int o = tpi / 2; o >= 1; o >>= 1) dot += __shfl_xor_sync(kAll, dot, o);
  if (dw != nullptr && live && in == 0) dw[item] = dot;
}

// -------------------------------------------------------------- on the grid
// The same flat range; a CTA takes `passes` runs of U vectors per thread.  The
// rows and gates of its tokens, which lie together, are looked up once into
// shared memory; in a pass a thread has the loads of KB choices (all of them,
// or 8 at a time) on the way before any is added.
constexpr uint32_t kLeastVectors = 8;    // per row, for the table to hold the tokens of one pass
constexpr uint32_t kTableEntries = 1024;
template <int DT, int VEC, int KB, int U>
__global__ void __launch_bounds__(kThreads) moe_from_experts_kernel(const __grid_constant__ MoeRowsArgs a, uint32_t nv, uint32_t passes) {
  constexpr int W = (VEC * Elem<DT>::kBytes + 3) / 4;
  static_assert((U * kThreads / kLeastVectors + 2) * (U > 1 ? KB : kMoeMaxK) <= kTableEntries, "the table holds a pass's choices");
  __shared__ int64_t first[kTableEntries];  // element of the row, or -1
  __shared__ float gate[kTableEntries];
  pdl_enter();
  const int r = blockIdx.y, k = a.k;
  const uint64_t total = static_cast<uint64_t>(a.tokens[r]) * nv;
  const uint64_t cta0 = static_cast<uint64_t>(blockIdx.x) * passes * (U * kThreads);
  if (cta0 >= total) return;
  const uint64_t cta1 = min(cta0 + static_cast<uint64_t>(passes) * (U * kThreads), total);
  const uint64_t t0 = split(cta0, nv).q, t1 = split(cta1 - 1, nv).q;
  const uint32_t entries = static_cast<uint32_t>(t1 - t0 + 1) * k;
  const float* weights = a.weights[r];
  for (uint32_t i = threadIdx.x; i < entries; i += kThreads) {
    const int64_t row = row_of(a.rows[r], t0 * k + i, a.cap[r]);
    first[i] = row >= 0 ? row * static_cast<int64_t>(a.hidden) : -1;
    gate[i] = weights != nullptr ? __ldg(weights + t0 * k + i) : 1.0f;
  }
  __syncthreads();
  // vectors from the first token's on: 32 bits serve
  const uint32_t f1 = static_cast<uint32_t>(cta1 - t0 * nv);
  for (uint32_t f0 = static_cast<uint32_t>(cta0 - t0 * nv) + threadIdx.x; f0 < f1; f0 += U * kThreads) {
    uint32_t token[U], v[U];
    float acc[U][VEC];
    bool have[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      token[u] = (f0 + u * kThreads) / nv;
      v[u] = (f0 + u * kThreads - token[u] * nv) * VEC;
      have[u] = false;
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[u][e] = -0.0f;  // -0 + x is x, to the bit
    }
    for (int j0 = 0; j0 < k; j0 += KB) {
      uint32_t raw[U][KB][W];
      bool there[U][KB];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int b = 0; b < KB; ++b) {
          const int64_t at = f0 + u * kThreads < f1 && j0 + b < k ? first[token[u] * k + j0 + b] : -1;
          there[u][b] = at >= 0;
          if (there[u][b]) load_raw<DT, VEC>(a.y[r], at + v[u], raw[u][b]);
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int b = 0; b < KB; ++b) {
          if (!there[u][b]) continue;
          const float wt = gate[token[u] * k + j0 + b];
#pragma unroll
          for (int e = 0; e < VEC; ++e) acc[u][e] = __fadd_rn(acc[u][e], __fmul_rn(wt, widen<DT>(raw[u][b], e)));
          have[u] = true;
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (f0 + u * kThreads >= f1) continue;
      if (!have[u]) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[u][e] = 0.0f;
      }
      uint32_t w[W];
      pack_out<DT, VEC>(acc[u], w);
      store_raw<DT, VEC>(a.out[r], (t0 + token[u]) * a.hidden + v[u], w);
    }
  }
}

// `tpt` threads (a power of two, 1..128) per token walk its vectors, U of them
// at a time: dout is read once for KB choices (all of them, or 8 at a time),
// each y vector once, each dy vector written once.  The dot products are added
// per thread, then in a fixed shuffle tree, then warp by warp.
template <int DT, int VEC, int KB, int U>
__global__ void __launch_bounds__(kThreads) moe_from_experts_grad_kernel(const __grid_constant__ MoeRowsArgs a,
                                                                        uint32_t nv, int tpt) {
  constexpr int W = (VEC * Elem<DT>::kBytes + 3) / 4;
  __shared__ float part[kThreads / 32][KB];
  pdl_enter();
  const int r = blockIdx.y, k = a.k;
  const int group = threadIdx.x / tpt, in = threadIdx.x - group * tpt, lane = threadIdx.x & 31;
  const uint64_t t = static_cast<uint64_t>(blockIdx.x) * (kThreads / tpt) + group;
  if (static_cast<uint64_t>(blockIdx.x) * (kThreads / tpt) >= a.tokens[r]) return;
  const bool live = t < a.tokens[r];
  const float* weights = a.weights[r];
  void* dy = a.out[r];
  float* dw = a.dweights[r];
  for (int j0 = 0; j0 < k; j0 += KB) {
    int64_t row[KB];
    float wt[KB], dot[KB];
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      row[b] = (live && j0 + b < k) ? row_of(a.rows[r], t * k + j0 + b, a.cap[r]) : -1;
      wt[b] = (live && weights != nullptr && j0 + b < k) ? __ldg(weights + t * k + j0 + b) : 1.0f;
      dot[b] = 0.0f;
    }
    for (uint32_t v0 = in; live && v0 < nv; v0 += tpt * U) {
      uint32_t d[U][W], y[U][KB][W];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t v = v0 + u * tpt;
        if (v >= nv) continue;
        load_raw<DT, VEC>(a.x[r], t * a.hidden + static_cast<uint64_t>(v) * VEC, d[u]);
        if (dw == nullptr) continue;
#pragma unroll
        for (int b = 0; b < KB; ++b)
          if (row[b] >= 0) load_raw<DT, VEC>(a.y[r], row[b] * a.hidden + static_cast<uint64_t>(v) * VEC, y[u][b]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t v = v0 + u * tpt;
        if (v >= nv) continue;
#pragma unroll
        for (int b = 0; b < KB; ++b) {
          if (row[b] < 0) continue;
          float o[VEC];
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float de = widen<DT>(d[u], e);
            o[e] = __fmul_rn(wt[b], de);
            if (dw != nullptr) dot[b] = fmaf(widen<DT>(y[u][b], e), de, dot[b]);
          }
          if (dy != nullptr) {
            uint32_t w[W];
            pack_out<DT, VEC>(o, w);
            store_raw<DT, VEC>(dy, row[b] * a.hidden + static_cast<uint64_t>(v) * VEC, w);
          }
        }
      }
    }
    if (dw == nullptr) continue;
    for (int o = (tpt < 32 ? tpt : 32) / 2; o >= 1; o >>= 1) {
#pragma unroll
      for (int b = 0; b < KB; ++b) dot[b] += __shfl_xor_sync(kAll, dot[b], o);
    }
    if (tpt <= 32) {
#pragma unroll
      for (int b = 0; b < KB; ++b)
        if (live && in == 0 && j0 + b < k) dw[t * k + j0 + b] = dot[b];
      continue;
    }
    if (lane == 0) {
#pragma unroll
      for (int b = 0; b < KB; ++b) part[threadIdx.x >> 5][b] = dot[b];
    }
    __syncthreads();
    if (live && in < KB && j0 + in < k) {
      float sum = 0.0f;
      for (int w = 0; w < tpt / 32; ++w) sum += part[group * (tpt / 32) + w][in];
      dw[t * k + j0 + in] = sum;
    }
    __syncthreads();
  }
}

uint32_t most_tokens(const MoeRowsArgs& a) {
  uint32_t m = 0;
  for (int r = 0; r < a.p; ++r) m = a.tokens[r] > m ? a.tokens[r] : m;
  return m;
}

template <typename... Params>
cudaError_t launch_rows(void (*kernel)(Params...), uint64_t ctas, int p, cudaStream_t s, Params... params) {
  if (ctas == 0) return cudaSuccess;  // no rank has a row to write
  if (ctas > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(p));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = CCL_PDL ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, params...);
  if (err == cudaSuccess) note_launch();
  return err;
}

cudaError_t launch_copy(int elem, const MoeRowsArgs& a, cudaStream_t s) {
  const uint32_t nv = static_cast<uint32_t>(a.hidden * elem / 16);
  const uint64_t total = static_cast<uint64_t>(most_tokens(a)) * nv, per = kThreads * kCopyVectors;
  return launch_rows(moe_to_experts_kernel, (total + per - 1) / per, a.p, s, a, nv);
}

uint64_t ctas_for(uint64_t threads) { return (threads + kThreads - 1) / kThreads; }

// The power of two of threads that walk `units` units, between lo and hi.
int walkers(uint64_t units, int lo, int hi) {
  int n = lo;
  while (n < hi && static_cast<uint64_t>(n) < units) n *= 2;
  return n;
}

template <int DT>
cudaError_t launch_back_grad_off(const MoeRowsArgs& a, cudaStream_t s) {
  const uint64_t row_bytes = a.hidden * Elem<DT>::kBytes;
  const int tpi = walkers(granules(row_bytes), 1, 32);
  const uint64_t per = kThreads / tpi, items = static_cast<uint64_t>(most_tokens(a)) * a.k;
  return launch_rows(moe_from_experts_grad_off_kernel<DT>, (items + per - 1) / per, a.p, s, a, row_bytes, tpi);
}

// Calls f(KB, U) with the choices that are loaded together and the vectors per
// thread.
template <typename F>
cudaError_t by_choices(int k, F f) {
  if (k == 1) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 2>{});
  if (k == 2) return f(std::integral_constant<int, 2>{}, std::integral_constant<int, 2>{});
  if (k <= 4) return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
  return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
}

template <int DT>
cudaError_t launch_back_off(const MoeRowsArgs& a, cudaStream_t s) {
  const uint64_t row_bytes = a.hidden * Elem<DT>::kBytes, ctas = ctas_for(most_tokens(a) * granules(row_bytes));
  return by_choices(a.k, [&](auto kb, auto) {
    return launch_rows(moe_from_experts_off_kernel<DT, decltype(kb)::value>, ctas, a.p, s, a, row_bytes);
  });
}

constexpr uint64_t kPassCtas = 4 * 152 * 4;  // waves, SMs, CTAs that an SM takes

template <int DT, int VEC>
cudaError_t launch_back(const MoeRowsArgs& a, cudaStream_t s) {
  const uint32_t nv = static_cast<uint32_t>(a.hidden / VEC);
  const uint64_t total = static_cast<uint64_t>(most_tokens(a)) * nv;
  return by_choices(a.k, [&](auto kb, auto u) {
    constexpr int KB = decltype(kb)::value, U = decltype(u)::value;
    // as many passes as leave four waves of CTAs (eight at most), and no more
    // than the table has room for
    const uint64_t pass = static_cast<uint64_t>(U) * kThreads;
    uint64_t passes = total * a.p / (pass * kPassCtas);
    const uint64_t room = (kTableEntries / a.k - 2) * nv / pass;
    passes = passes > 8 ? 8 : passes;
    passes = passes > room ? room : passes;
    if (passes == 0) passes = 1;
    return launch_rows(moe_from_experts_kernel<DT, VEC, KB, U>, (total + pass * passes - 1) / (pass * passes), a.p, s, a, nv,
                       static_cast<uint32_t>(passes));
  });
}

// At most 128 threads a token: 8 ranks x 2048 tokens x 7168 bf16 of 8 choices
// took 631 us with 256, 597 with 128 or 64, 601 with 32.
template <int DT, int VEC>
cudaError_t launch_back_grad(const MoeRowsArgs& a, cudaStream_t s) {
  const uint32_t nv = static_cast<uint32_t>(a.hidden / VEC);
  return by_choices(a.k, [&](auto kb, auto u) {
    constexpr int KB = decltype(kb)::value, U = KB == 1 ? 4 : decltype(u)::value;
    const int tpt = walkers((nv + U - 1) / U, 1, 128);
    const uint64_t per = kThreads / tpt;
    return launch_rows(moe_from_experts_grad_kernel<DT, VEC, KB, U>, (most_tokens(a) + per - 1) / per, a.p, s, a, nv, tpt);
  });
}

}  // namespace

cudaError_t launch_moe_sort(const MoeSortArgs& a, cudaStream_t s) {
  uint32_t most = 0;
  for (int r = 0; r < a.p; ++r) most = a.items[r] > most ? a.items[r] : most;
  // CTAs of few warps before warps: the votes fill a SM's issue slots (4096
  // items of 256 experts 3.3 us in 4 CTAs of 8 warps, 4.3 in 2 of 16, 6.8 in one
  // of 32), and columns of few warps are short.  Once the cluster has 16 CTAs,
  // up to 32 warps each.
  constexpr uint32_t kLeastWarps = 8, kPerCta = kPerTurn * kLeastWarps;
  const uint32_t wanted = (most + kPerCta - 1) / kPerCta, ctas = wanted < 1 ? 1 : wanted > kSortMaxCluster ? kSortMaxCluster : wanted;
  uint32_t warps = ((most + ctas * kPerTurn - 1) / (ctas * kPerTurn) + 7) / 8 * 8;
  warps = warps < 8 ? 8 : warps > kSortMaxWarps ? kSortMaxWarps : warps;
  const size_t smem = (static_cast<size_t>(warps) + 2) * a.num_experts * sizeof(uint32_t);
  // The limits belong to the function, not to the call: always the most that a
  // call may need, so that host threads cannot lower each other's between the
  // setting and the launch.
  constexpr int kMostSmem = (kSortMaxWarps + 2) * kSortMaxExperts * sizeof(uint32_t);
  cudaError_t err = cudaSuccess;
  if (ctas > 8) err = cudaFuncSetAttribute(moe_sort_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (err == cudaSuccess && smem > 48 * 1024) err = cudaFuncSetAttribute(moe_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, static_cast<unsigned>(a.p));
  cfg.blockDim = dim3(warps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = CCL_PDL ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  err = cudaLaunchKernelEx(&cfg, moe_sort_kernel, a);
  if (err == cudaSuccess) note_launch();
  return err;
}

cudaError_t launch_moe_to_experts(int dt, bool vec, const MoeRowsArgs& a, cudaStream_t s) {
  const int elem = dt == kF32 ? 4 : 2;
  if (vec) return launch_copy(elem, a, s);
  const uint64_t row_bytes = a.hidden * elem, ctas = ctas_for((static_cast<uint64_t>(most_tokens(a)) * a.k * granules(row_bytes) + kOffUnits - 1) / kOffUnits);
  return elem == 4 ? launch_rows(moe_to_experts_off_kernel<4>, ctas, a.p, s, a, row_bytes)
                   : launch_rows(moe_to_experts_off_kernel<2>, ctas, a.p, s, a, row_bytes);
}

cudaError_t launch_moe_from_experts(int dt, bool vec, const MoeRowsArgs& a, cudaStream_t s) {
  // rows of fewer vectors than the table allows go by granules too
  if (dt == kF32) return vec && a.hidden >= 4 * kLeastVectors ? launch_back<kF32, 4>(a, s) : launch_back_off<kF32>(a, s);
  return vec && a.hidden >= 8 * kLeastVectors ? launch_back<kBF16, 8>(a, s) : launch_back_off<kBF16>(a, s);
}

cudaError_t launch_moe_from_experts_grad(int dt, bool vec, const MoeRowsArgs& a, cudaStream_t s) {
  if (dt == kF32) return vec ? launch_back_grad<kF32, 4>(a, s) : launch_back_grad_off<kF32>(a, s);
  return vec ? launch_back_grad<kBF16, 8>(a, s) : launch_back_grad_off<kBF16>(a, s);
}

}  // namespace ccl
