// norm.cu -- layer norm over rows, and its gradients.
//
//   v = x (+ residual, rounded to the rows' type), m = mean(v),
//   s = (mean((v - m)^2) + eps)^-1/2,  y = (v - m) s w + b;
//   with z = (v - m) s and g = dy w:
//   dx = s (g - mean(g) - z mean(g z)) + dsum,  dw = sum over rows of dy z,  db = of dy.
//
// Rows move once in each direction, so HBM bounds all of it.  A group of one or
// more warps has a row; a thread has the same columns of every row that its
// group takes, so that the sums over rows stay in its registers.
#include "row_parts.cuh"

namespace ccl {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;

// N consecutive elements at `base` + i as floats: by one load where they are 16
// bytes, by 16-byte loads where they are more.
template <int DT, int N>
__device__ __forceinline__ void widen_raw(const uint32_t* w, float* f) {
#pragma unroll
  for (int e = 0; e < N; ++e) f[e] = widen<DT>(w, e);
}

// The weights of N columns.  They are read again for every row and stay in L1.
// `grid`: on 16 bytes, as N columns' bytes are.
template <int WT, int N>
__device__ __forceinline__ void load_weights(const void* base, uint32_t c, bool grid, float* f) {
  constexpr int B = Elem<WT>::kBytes;
  const char* p = static_cast<const char*>(base) + static_cast<size_t>(c) * B;
  if (N * B >= 16 && grid) {
    uint32_t w[N * B >= 16 ? N * B / 4 : 4];
#pragma unroll
    for (int k = 0; k < N * B / 16; ++k) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[k];
      w[4 * k] = v.x;
      w[4 * k + 1] = v.y;
      w[4 * k + 2] = v.z;
      w[4 * k + 3] = v.w;
    }
    widen_raw<WT, N>(w, f);
  } else if (N * B == 8 && grid) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    const uint32_t w[2] = {v.x, v.y};
    widen_raw<WT, N>(w, f);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if constexpr (WT == kF32) f[e] = reinterpret_cast<const float*>(p)[e];
      else f[e] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[e]);
    }
  }
}

// ------------------------------------------------------------ groups of warps
// Sums over a group, the same for every thread and in a fixed order: by
// shuffles within the warps, then through shared memory in two sets of slots
// in turn, so that one barrier of the group does for each sum.
constexpr int kMostWarps = 32;  // of a CTA
struct Group {
  int warps, warp, lane, id;  // warps of the group, this one among them, the group's number
  int turn = 0;
  float4* slots;              // 2 x kMostWarps
  __device__ __forceinline__ Group(float4* s, int group_threads) {
    warps = group_threads >> 5;
    id = static_cast<int>(threadIdx.x) / group_threads;
    warp = (static_cast<int>(threadIdx.x) - id * group_threads) >> 5;
    lane = threadIdx.x & 31;
    slots = s;
  }
  __device__ __forceinline__ void sync() const {
    asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(warps * 32) : "memory");
  }
  template <int N>
  __device__ __forceinline__ void sum(float* v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(kAll, v[i], o);
    if (warps == 1) return;
    float4* s = slots + turn * kMostWarps + id * warps;
    turn ^= 1;
    if (lane == 0) s[warp] = make_float4(v[0], N > 1 ? v[N > 1 ? 1 : 0] : 0.f, N > 2 ? v[N > 2 ? 2 : 0] : 0.f, N > 3 ? v[N > 3 ? 3 : 0] : 0.f);
    sync();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
    for (int w = 0; w < warps; ++w) {
      const float4 t = s[w];
      v[0] += t.x;
      if (N > 1) v[N > 1 ? 1 : 0] += t.y;
      if (N > 2) v[N > 2 ? 2 : 0] += t.z;
      if (N > 3) v[N > 3 ? 3 : 0] += t.w;
    }
  }
};

// -------------------------------------------------------------------- forward
// The row stays in registers between its three walks (mean, variance, output).
// VEC elements are 16 bytes on the grid, one element off it; a thread has U
// such units.
template <int DT, int WT, int VEC, int U, bool SUM>
__global__ void __launch_bounds__(512) norm_kernel(const __grid_constant__ NormArgs a, int group_threads, uint32_t weights_on_grid) {
  constexpr int WORDS = VEC * Elem<DT>::kBytes >= 4 ? VEC * Elem<DT>::kBytes / 4 : 1;
  __shared__ float4 slots[2 * kMostWarps];
  pdl_enter();
  Group group(slots, group_threads);
  const RowPart part = row_part(a.parts, a.p, blockIdx.x);
  const int r = part.r, groups = blockDim.x / group_threads, t = threadIdx.x - group.id * group_threads;
  const uint32_t cols = a.cols, units = cols / VEC;
  const float n = static_cast<float>(cols), eps = static_cast<float>(a.eps);
  for (uint32_t row = part.lo + group.id; row < part.hi; row += groups) {
    const uint64_t at = static_cast<uint64_t>(row) * cols;
    uint32_t w[U][WORDS];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t u = t + i * group_threads;
#pragma unroll
      for (int k = 0; k < WORDS; ++k) w[i][k] = 0;
      if (u < units) load_raw<DT, VEC>(a.x[r], at + u * VEC, w[i]);
    }
    if constexpr (SUM) {
      uint32_t q[U][WORDS];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const uint32_t u = t + i * group_threads;
#pragma unroll
        for (int k = 0; k < WORDS; ++k) q[i][k] = 0;
        if (u < units) load_raw<DT, VEC>(a.extra[r], at + u * VEC, q[i]);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const uint32_t u = t + i * group_threads;
        float f[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = widen<DT>(w[i], e) + widen<DT>(q[i], e);
        pack_out<DT, VEC>(f, w[i]);
        if (u < units) store_raw<DT, VEC>(a.sum[r], at + u * VEC, w[i]);
      }
    }
    float total[1] = {0.f};
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) total[0] += widen<DT>(w[i], e);
    group.sum<1>(total);
    const float mean = total[0] / n;
    float square[1] = {0.f};
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t u = t + i * group_threads;
      if (u >= units) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = widen<DT>(w[i], e) - mean;
        square[0] = fmaf(d, d, square[0]);
      }
    }
    group.sum<1>(square);
    const float rstd = 1.f / sqrtf(square[0] / n + eps);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t u = t + i * group_threads;
      if (u >= units) continue;
      float scale[VEC], shift[VEC], f[VEC];
      load_weights<WT, VEC>(a.weight[r], u * VEC, weights_on_grid, scale);
      if (a.bias[r] != nullptr) load_weights<WT, VEC>(a.bias[r], u * VEC, weights_on_grid, shift);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if (a.bias[r] == nullptr) shift[e] = 0.f;
        f[e] = fmaf((widen<DT>(w[i], e) - mean) * rstd, scale[e], shift[e]);
      }
      uint32_t o[WORDS];
      pack_out<DT, VEC>(f, o);
      store_raw<DT, VEC>(a.out[r], at + u * VEC, o);
    }
    if (t == 0 && a.mean[r] != nullptr) {
      a.mean[r][row] = mean;
      a.rstd[r][row] = rstd;
    }
  }
}

// ------------------------------------------------------------------- backward
// The sums over rows of a CTA's groups, group after group, to its part.
template <int VEC, int U>
__device__ __forceinline__ void write_part(const NormArgs& a, const Group& group, int groups, int group_threads, float* shared,
                                           const float (&dw)[U][VEC], const float (&db)[U][VEC]) {
  if (a.partial == nullptr) return;
  const uint32_t cols = a.cols;
  const int t = threadIdx.x - group.id * group_threads;
  float* out = a.partial + static_cast<uint64_t>(blockIdx.x) * 2 * cols;
  // all but the last group through shared memory
  for (int g = 0; g < groups; ++g) {
    __syncthreads();
    if (g != group.id) continue;
    float* to = g == groups - 1 ? out : shared;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t c = (t + i * group_threads) * VEC;
      if (c >= cols) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        to[c + e] = g == 0 ? dw[i][e] : shared[c + e] + dw[i][e];
        to[cols + c + e] = g == 0 ? db[i][e] : shared[cols + c + e] + db[i][e];
      }
    }
  }
}

__device__ __forceinline__ void copy16_async(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// Rows on the 16-byte grid.  R rows at a time come through a ring in shared
// memory of `depth` stages, in which each thread copies what it reads itself, so
// that no barrier stands between the copies and their use; both walks over a
// row (sums, then output) read it there.
template <int DT, int WT, int U, int R, bool EXTRA>
__global__ void __launch_bounds__(512) norm_grad_kernel(const __grid_constant__ NormArgs a, int group_threads, int depth, uint32_t weights_on_grid) {
  constexpr int VEC = 16 / Elem<DT>::kBytes, ARRAYS = EXTRA ? 3 : 2, PER_STAGE = R * ARRAYS * U;
  extern __shared__ uint4 ring[];  // [depth][R][ARRAYS][U][threads]
  __shared__ float4 slots[2 * kMostWarps];
  pdl_enter();
  Group group(slots, group_threads);
  const RowPart part = row_part(a.parts, a.p, blockIdx.x);
  const int r = part.r, groups = blockDim.x / group_threads, t = threadIdx.x - group.id * group_threads;
  const uint32_t cols = a.cols, units = cols / VEC;
  const float inv = 1.f / static_cast<float>(cols);
  const uint4* mine = ring + threadIdx.x;
  const uint32_t mine_at = static_cast<uint32_t>(__cvta_generic_to_shared(mine)), step = blockDim.x * 16;
  float dw[U][VEC], db[U][VEC];
#pragma unroll
  for (int i = 0; i < U; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[i][e] = db[i][e] = 0.f;

  const auto fetch = [&](uint64_t row0, int stage) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (row0 + j >= part.hi) break;
      const uint64_t at = (row0 + j) * cols;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const uint32_t u = t + i * group_threads;
        if (u >= units) break;
        const uint64_t byte = (at + u * VEC) * Elem<DT>::kBytes;
        const uint32_t to = mine_at + (stage * PER_STAGE + j * ARRAYS * U + i) * step;
        copy16_async(to, static_cast<const char*>(a.x[r]) + byte);
        copy16_async(to + U * step, static_cast<const char*>(a.dy[r]) + byte);
        if constexpr (EXTRA) copy16_async(to + 2 * U * step, static_cast<const char*>(a.extra[r]) + byte);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const uint64_t stride = static_cast<uint64_t>(groups) * R;
  uint64_t ahead = part.lo + static_cast<uint64_t>(group.id) * R, row0 = ahead;
  for (int d = 0; d < depth - 1; ++d, ahead += stride) fetch(ahead, d);
  float mean[R], rstd[R];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const bool there = row0 + j < part.hi;
    mean[j] = there ? a.mean[r][row0 + j] : 0.f;
    rstd[j] = there ? a.rstd[r][row0 + j] : 0.f;
  }
  for (int stage = 0; row0 < part.hi; row0 += stride) {
    {
      int next = stage + depth - 1;
      fetch(ahead, next >= depth ? next - depth : next);
      ahead += stride;
    }
    float next_mean[R], next_rstd[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const bool there = row0 + stride + j < part.hi;
      next_mean[j] = there ? a.mean[r][row0 + stride + j] : 0.f;
      next_rstd[j] = there ? a.rstd[r][row0 + stride + j] : 0.f;
    }
    if (depth == 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (depth == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else asm volatile("cp.async.wait_group 1;" ::: "memory");
    const uint4* here = mine + stage * PER_STAGE * blockDim.x;
    float sums[2 * R];
#pragma unroll
    for (int j = 0; j < 2 * R; ++j) sums[j] = 0.f;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t u = t + i * group_threads;
      if (u >= units) break;
      float weight[VEC];
      load_weights<WT, VEC>(a.weight[r], u * VEC, weights_on_grid, weight);
#pragma unroll
      for (int j = 0; j < R; ++j) {
        if (row0 + j >= part.hi) break;
        const uint4 xv = here[(j * ARRAYS * U + i) * blockDim.x], dv = here[(j * ARRAYS * U + U + i) * blockDim.x];
        const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w}, dyw[4] = {dv.x, dv.y, dv.z, dv.w};
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float z = (widen<DT>(xw, e) - mean[j]) * rstd[j], d = widen<DT>(dyw, e), g = d * weight[e];
          sums[2 * j] += g;
          sums[2 * j + 1] = fmaf(g, z, sums[2 * j + 1]);
          dw[i][e] = fmaf(d, z, dw[i][e]);
          db[i][e] += d;
        }
      }
    }
    group.sum<2 * R>(sums);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t u = t + i * group_threads;
      if (u >= units) break;
      float weight[VEC];
      load_weights<WT, VEC>(a.weight[r], u * VEC, weights_on_grid, weight);
#pragma unroll
      for (int j = 0; j < R; ++j) {
        if (row0 + j >= part.hi) break;
        const uint4 xv = here[(j * ARRAYS * U + i) * blockDim.x], dv = here[(j * ARRAYS * U + U + i) * blockDim.x];
        const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w}, dyw[4] = {dv.x, dv.y, dv.z, dv.w};
        uint4 ev = make_uint4(0, 0, 0, 0);
        if constexpr (EXTRA) ev = here[(j * ARRAYS * U + 2 * U + i) * blockDim.x];
        const uint32_t ew[4] = {ev.x, ev.y, ev.z, ev.w};
        const float mg = sums[2 * j] * inv, mgz = sums[2 * j + 1] * inv;
        float f[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float z = (widen<DT>(xw, e) - mean[j]) * rstd[j];
          f[e] = (fmaf(widen<DT>(dyw, e), weight[e], -mg) - z * mgz) * rstd[j];
          if constexpr (EXTRA) f[e] += widen<DT>(ew, e);
        }
        uint32_t o[4];
        pack_out<DT, VEC>(f, o);
        store_raw<DT, VEC>(a.out[r], (row0 + j) * cols + u * VEC, o);
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      mean[j] = next_mean[j];
      rstd[j] = next_rstd[j];
    }
    stage = stage + 1 == depth ? 0 : stage + 1;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  write_part<VEC, U>(a, group, groups, group_threads, reinterpret_cast<float*>(ring), dw, db);
}

// Rows off the grid, or too long for a ring: element by element; the second walk
// finds the row in L1 or L2.
template <int DT, int WT, int U>
__global__ void __launch_bounds__(512) norm_grad_off_kernel(const __grid_constant__ NormArgs a, int group_threads) {
  extern __shared__ uint4 ring[];
  __shared__ float4 slots[2 * kMostWarps];
  pdl_enter();
  Group group(slots, group_threads);
  const RowPart part = row_part(a.parts, a.p, blockIdx.x);
  const int r = part.r, groups = blockDim.x / group_threads, t = threadIdx.x - group.id * group_threads;
  const uint32_t cols = a.cols;
  const float inv = 1.f / static_cast<float>(cols);
  float dw[U][1], db[U][1];
#pragma unroll
  for (int i = 0; i < U; ++i) dw[i][0] = db[i][0] = 0.f;
  const auto one = [](const void* base, uint64_t i) {
    if constexpr (DT == kF32) return static_cast<const float*>(base)[i];
    else return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i]);
  };
  for (uint64_t row = part.lo + static_cast<uint64_t>(group.id); row < part.hi; row += groups) {
    const uint64_t at = row * cols;
    const float mean = a.mean[r][row], rstd = a.rstd[r][row];
    float sums[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t c = t + i * group_threads;
      if (c >= cols) break;
      float weight;
      load_weights<WT, 1>(a.weight[r], c, false, &weight);
      const float z = (one(a.x[r], at + c) - mean) * rstd, d = one(a.dy[r], at + c), g = d * weight;
      sums[0] += g;
      sums[1] = fmaf(g, z, sums[1]);
      dw[i][0] = fmaf(d, z, dw[i][0]);
      db[i][0] += d;
    }
    group.sum<2>(sums);
    const float mg = sums[0] * inv, mgz = sums[1] * inv;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t c = t + i * group_threads;
      if (c >= cols) break;
      float weight;
      load_weights<WT, 1>(a.weight[r], c, false, &weight);
      const float z = (one(a.x[r], at + c) - mean) * rstd;
      float f = (fmaf(one(a.dy[r], at + c), weight, -mg) - z * mgz) * rstd;
      if (a.extra[r] != nullptr) f += one(a.extra[r], at + c);
      uint32_t o;
      pack_out<DT, 1>(&f, &o);
      store_raw<DT, 1>(a.out[r], at + c, &o);
    }
  }
  write_part<1, U>(a, group, groups, group_threads, reinterpret_cast<float*>(ring), dw, db);
}

// A rank's parts added up: a CTA has 32 columns (grid y = rank), each of its warps
// every eighth part, and the warps' sums are added in order.
constexpr int kJoinWarps = 8;
template <int DT>
__global__ void __launch_bounds__(32 * kJoinWarps) norm_join_kernel(const __grid_constant__ NormJoinArgs a) {
  __shared__ float sums[2][kJoinWarps][32];
  pdl_enter();
  const int r = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t c = blockIdx.x * 32 + lane;
  float w = 0.f, b = 0.f;
  if (c < a.cols) {
#pragma unroll 4
    for (uint32_t i = a.first[r] + warp; i < a.first[r + 1]; i += kJoinWarps) {
      const float* part = a.partial + static_cast<uint64_t>(i) * 2 * a.cols;
      w += part[c];
      b += part[a.cols + c];
    }
  }
  sums[0][warp][lane] = w;
  sums[1][warp][lane] = b;
  __syncthreads();
  if (warp > 1 || c >= a.cols || !(warp == 0 ? a.weight : a.bias)) return;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) s += sums[warp][i][lane];
  uint32_t o;
  pack_out<DT, 1>(&s, &o);
  store_raw<DT, 1>(warp == 0 ? a.dweight[r] : a.dbias[r], c, &o);
}

// ------------------------------------------------------------------ launches
template <typename F>
cudaError_t by_types(int dt, int wt, F f) {
  const auto with = [&](auto d) {
    return wt == kF32 ? f(d, std::integral_constant<int, kF32>{}) : f(d, std::integral_constant<int, kBF16>{});
  };
  return dt == kF32 ? with(std::integral_constant<int, kF32>{}) : with(std::integral_constant<int, kBF16>{});
}
template <int N>
using Int = std::integral_constant<int, N>;

int whole_warps(uint32_t units, int per_thread) { return static_cast<int>((units + 32 * per_thread - 1) / (32 * per_thread)) * 32; }

template <typename... P, typename... A>
cudaError_t launch_norm_kernel(void (*kernel)(P...), uint32_t ctas, int threads, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = CCL_PDL ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (err == cudaSuccess) note_launch();
  return err;
}

// Whether every weight (and bias) starts on 16 bytes.
uint32_t weights_on_grid(const NormArgs& a) {
  uintptr_t bits = 0;
  for (int r = 0; r < a.p; ++r) bits |= reinterpret_cast<uintptr_t>(a.weight[r]) | reinterpret_cast<uintptr_t>(a.bias[r]);
  return (bits & 15) == 0;
}

}  // namespace

cudaError_t launch_norm(int dt, int weight_dt, bool vec, const NormArgs& args, cudaStream_t s) {
  const uint32_t grid = weights_on_grid(args);
  NormArgs a = args;
  size_t rows[kMoeMaxRanks];
  bool sum = false;
  for (int r = 0; r < a.p; ++r) {
    rows[r] = a.parts.rows[r];
    sum = sum || a.sum[r] != nullptr;
  }
  return by_types(dt, weight_dt, [&](auto d, auto w) {
    constexpr int DT = decltype(d)::value, WT = decltype(w)::value;
    const auto go = [&](auto ve, auto un) {
      constexpr int VEC = decltype(ve)::value, U = decltype(un)::value;
      const int group = whole_warps(a.cols / VEC, U), groups = group >= 256 ? 1 : 256 / group;
      // parts small enough that the last ones of a launch end together
      cut_rows(&a.parts, rows, a.p, 152 * 32, groups, false);
      return launch_norm_kernel(sum ? norm_kernel<DT, WT, VEC, U, true> : norm_kernel<DT, WT, VEC, U, false>, a.parts.first[a.p], group * groups, 0, s,
                                a, group, grid);
    };
    if (vec) {
      constexpr int VEC = 16 / Elem<DT>::kBytes;
      const uint32_t units = a.cols / VEC;
      if (units <= 32) return go(Int<VEC>{}, Int<1>{});
      if (units <= 64) return go(Int<VEC>{}, Int<2>{});
      return units <= 2048 ? go(Int<VEC>{}, Int<4>{}) : go(Int<VEC>{}, Int<8>{});
    }
    if (a.cols <= 128) return go(Int<1>{}, Int<4>{});
    return a.cols <= 8192 ? go(Int<1>{}, Int<16>{}) : go(Int<1>{}, Int<32>{});
  });
}

cudaError_t launch_norm_grad(int dt, int weight_dt, bool vec, NormArgs* args, cudaStream_t s) {
  constexpr size_t kMostRing = 216 * 1024;  // of a SM's shared memory
  NormArgs& a = *args;
  const uint32_t grid = weights_on_grid(a);
  size_t rows[kMoeMaxRanks];
  bool extra = false;
  for (int r = 0; r < a.p; ++r) {
    rows[r] = a.parts.rows[r];
    extra = extra || a.extra[r] != nullptr;
  }
  return by_types(dt, weight_dt, [&](auto d, auto w) {
    constexpr int DT = decltype(d)::value, WT = decltype(w)::value, VEC = 16 / Elem<DT>::kBytes;
    const auto launch = [&](auto* kernel, uint32_t ctas, int group, int groups, int at_once, size_t smem, auto... more) {
      cut_rows(&a.parts, rows, a.p, ctas, static_cast<uint32_t>(groups) * at_once, false);
      // the limit belongs to the function, not to the call: always the most that a call may need
      const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMostRing));
      if (err != cudaSuccess) return err;
      return launch_norm_kernel(kernel, a.parts.first[a.p], group * groups, smem, s, static_cast<const NormArgs&>(a), group, more...);
    };
    const auto off = [&](auto un) {
      constexpr int U = decltype(un)::value;
      const int group = whole_warps(a.cols, U), groups = group >= 256 ? 1 : 256 / group;
      return launch(norm_grad_off_kernel<DT, WT, U>, kNormParts, group, groups, 1, groups > 1 ? a.cols * 8 : 0);
    };
    const auto any_off = [&] {
      if (a.cols <= 128) return off(Int<4>{});
      return a.cols <= 8192 ? off(Int<16>{}) : off(Int<32>{});
    };
    // as many groups of up to 512 threads as leave room for two stages; false where not even one does
    cudaError_t err = cudaSuccess;
    const auto on = [&](auto un, auto rs) {
      constexpr int U = decltype(un)::value, R = decltype(rs)::value;
      const int group = whole_warps(a.cols / VEC, U);
      const size_t stage = static_cast<size_t>(group) * 16 * R * (extra ? 3 : 2) * U;
      const size_t fit = kMostRing / (2 * stage), most = group >= 512 ? 1 : 512 / group;
      if (fit == 0) return false;
      const int groups = static_cast<int>(fit < most ? fit : most);
      const size_t room = kMostRing / (groups * stage), parts = groups > 1 ? a.cols * 8 : 0;
      const int depth = static_cast<int>(room > 4 ? 4 : room);
      const size_t ring = depth * groups * stage, smem = ring > parts ? ring : parts;
      // a CTA a SM, two of the small ones
      const uint32_t ctas = U * VEC <= 8 && 2 * smem <= kMostRing ? kNormParts : kNormParts / 2;
      err = launch(extra ? norm_grad_kernel<DT, WT, U, R, true> : norm_grad_kernel<DT, WT, U, R, false>, ctas, group, groups, R, smem, depth, grid);
      return true;
    };
    constexpr int U8 = 8 / VEC, U16 = 16 / VEC, U32 = 32 / VEC;
    const bool done = vec && (a.cols <= 256    ? on(Int<U8>{}, Int<1>{})
                              : a.cols <= 512  ? on(Int<U16>{}, Int<1>{})
                              : a.cols <= 1024 ? on(Int<U32>{}, Int<1>{})
                              : a.cols <= 8192 ? on(Int<U16>{}, Int<2>{}) || on(Int<U16>{}, Int<1>{})
                                               : on(Int<U32>{}, Int<1>{}));
    return done ? err : any_off();
  });
}

cudaError_t launch_norm_join(int dw_dt, const NormJoinArgs& a, cudaStream_t s) {
  const dim3 grid((a.cols + 31) / 32, static_cast<unsigned>(a.p));
  const cudaError_t err = dw_dt == kF32 ? launch_kernel(norm_join_kernel<kF32>, grid, dim3(32 * kJoinWarps), s, a)
                                        : launch_kernel(norm_join_kernel<kBF16>, grid, dim3(32 * kJoinWarps), s, a);
  if (err == cudaSuccess) note_launch();
  return err;
}

}  // namespace ccl
