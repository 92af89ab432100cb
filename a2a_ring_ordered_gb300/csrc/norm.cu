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
#include "pairs.cuh"
#include "realign.cuh"
#include "row_parts.cuh"

namespace ccl {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;

// ------------------------------------------------------------------- units
// A row goes in units of 16 bytes from its start, thread t of a group having units
// t, t + threads, ...: the same columns in every row.  GRID: all rows start on 16
// bytes and are whole units.  Off the grid a unit is cut out of the two aligned
// granules that hold it, the last unit may be part of one, and aligned granules
// are put together from neighbouring lanes' units for the stores.
template <int DT, bool GRID>
struct Units {
  static constexpr int kBytes = Elem<DT>::kBytes, kPer = 16 / kBytes;
  uint32_t row_bytes, count;
  __device__ __forceinline__ explicit Units(uint32_t cols) : row_bytes(cols * kBytes), count((row_bytes + 15) / 16) {}
  // The unit's bytes that are the row's.
  __device__ __forceinline__ uint32_t bytes(uint32_t u) const {
    if (GRID) return u < count ? 16 : 0;
    return u < count ? min(16u, row_bytes - 16 * u) : 0;
  }
  // The unit, zeros where it is not the row's.
  __device__ __forceinline__ uint4 load(const char* row, uint32_t u) const {
    if constexpr (GRID) return u < count ? ld_once16(row + 16 * u) : make_uint4(0, 0, 0, 0);
    const uint32_t n = bytes(u);
    const uint4 v = load16_part(row + 16 * u, 0, n);
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) w[k] = n >= 4 * k + 4 ? w[k] : n == 4 * k + 2 ? w[k] & 0xFFFFu : 0;
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // All lanes of a warp together.
  __device__ __forceinline__ void store(char* row, uint32_t u, const uint32_t* w) const {
    const uint4 v = make_uint4(w[0], w[1], w[2], w[3]);
    const uint32_t n = bytes(u), phase = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row)) & 15;
    char* to = row + 16 * u;
    if constexpr (GRID) {
      if (n) st_stream16(to, v);
      return;
    }
    // `first` bytes of the unit lie in its first granule; the second one takes the rest and the next lane's first
    const int lane = threadIdx.x & 31;
    const uint32_t first = 16 - phase;
    const uint4 next = next_lane(v, make_uint4(0, 0, 0, 0), lane);
    const uint32_t next_n = __shfl_down_sync(kAll, n, 1);
    const bool whole = n == 16 && (phase == 0 || (lane < 31 && next_n >= first));
    if (whole) st_stream16(phase == 0 ? to : to + first, phase == 0 ? v : shift16(v, next, first));
    // what no lane's granule holds
    const bool head = phase != 0 && (lane == 0 || n < first);
    if (!head && whole) return;
#pragma unroll
    for (uint32_t e = 0; e < kPer; ++e) {
      const uint32_t at = e * kBytes;
      if (at < n && (phase != 0 && at < first ? head : !whole)) store_one<DT>(to, e, w, e);
    }
  }
};

// The weights of the N columns from c on, zeros from cols on; they are read again
// for every row and stay in L1.  `grid`: their columns start on 16 bytes.
template <int WT, int N>
__device__ __forceinline__ void load_weights(const void* base, uint32_t c, uint32_t cols, bool grid, F2* f) {
  constexpr int B = Elem<WT>::kBytes, kWords = N * B / 4;
  const char* p = static_cast<const char*>(base) + static_cast<size_t>(c) * B;
  uint32_t w[kWords];
  if (grid && c + N <= cols) {
    if constexpr (kWords >= 4) {
#pragma unroll
      for (int k = 0; k < kWords / 4; ++k) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[k];
        w[4 * k] = v.x;
        w[4 * k + 1] = v.y;
        w[4 * k + 2] = v.z;
        w[4 * k + 3] = v.w;
      }
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x;
      w[1] = v.y;
    }
  } else {
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if (c + e >= cols) continue;
      if constexpr (WT == kF32) w[e] = reinterpret_cast<const uint32_t*>(p)[e];
      else w[e / 2] |= static_cast<uint32_t>(reinterpret_cast<const unsigned short*>(p)[e]) << (16 * (e & 1));
    }
  }
#pragma unroll
  for (int i = 0; i < N / 2; ++i) f[i] = widen2<WT>(w, i);
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
template <int DT, int WT, int U, bool SUM, bool GRID>
__global__ void __maxnreg__(U <= 2 ? 64 : U == 4 ? 80 : 128) norm_kernel(const __grid_constant__ NormArgs a, int group_threads, uint32_t weights_on_grid) {
  constexpr int VEC = 16 / Elem<DT>::kBytes, P = VEC / 2;
  __shared__ float4 slots[2 * kMostWarps];
  pdl_enter();
  Group group(slots, group_threads);
  const RowPart part = row_part(a.parts, a.p, blockIdx.x);
  const int r = part.r, groups = blockDim.x / group_threads, t = threadIdx.x - group.id * group_threads;
  const uint32_t cols = a.cols;
  const Units<DT, GRID> units(cols);
  const float n = static_cast<float>(cols), eps = static_cast<float>(a.eps);
  const char *x = static_cast<const char*>(a.x[r]), *extra = static_cast<const char*>(a.extra[r]);
  for (uint32_t row = part.lo + group.id; row < part.hi; row += groups) {
    const uint64_t at = static_cast<uint64_t>(row) * units.row_bytes;
    F2 f[U][P];
    {
      uint4 v[U];
#pragma unroll
      for (int i = 0; i < U; ++i) v[i] = units.load(x + at, t + i * group_threads);
      if constexpr (SUM) {
        uint4 q[U];
#pragma unroll
        for (int i = 0; i < U; ++i) q[i] = units.load(extra + at, t + i * group_threads);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w}, o[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
          if constexpr (DT == kBF16) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __nv_bfloat162 h = __hadd2(*reinterpret_cast<__nv_bfloat162*>(&w[k]), *reinterpret_cast<__nv_bfloat162*>(&o[k]));
              w[k] = *reinterpret_cast<const uint32_t*>(&h);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = __float_as_uint(__uint_as_float(w[k]) + __uint_as_float(o[k]));
          }
          units.store(static_cast<char*>(a.sum[r]) + at, t + i * group_threads, w);
          v[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int k = 0; k < P; ++k) f[i][k] = widen2<DT>(w, k);
      }
    }
    F2 sum = both(0.f);
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int k = 0; k < P; ++k) sum = add2(sum, f[i][k]);
    float total[1] = {total2(sum)};
    group.sum<1>(total);
    const float mean = total[0] / n;
    const F2 less = both(-mean);
    sum = both(0.f);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t left = units.bytes(t + i * group_threads) / Elem<DT>::kBytes;  // elements of the unit
#pragma unroll
      for (int k = 0; k < P; ++k) {
        f[i][k] = add2(f[i][k], less);
        if (GRID) {
          if (left == 0) f[i][k] = both(0.f);
        } else {
          const float2 d = parts(f[i][k]);
          f[i][k] = pair(left > 2 * k ? d.x : 0.f, left > 2 * k + 1 ? d.y : 0.f);
        }
        sum = fma2(f[i][k], f[i][k], sum);
      }
    }
    float square[1] = {total2(sum)};
    group.sum<1>(square);
    const float rstd = 1.f / sqrtf(square[0] / n + eps);
    const F2 scale = both(rstd);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t u = t + i * group_threads;
      if (GRID && u >= units.count) break;
      F2 w[P], b[P];
      load_weights<WT, VEC>(a.weight[r], u * VEC, cols, weights_on_grid, w);
      if (a.bias[r] != nullptr) {
        load_weights<WT, VEC>(a.bias[r], u * VEC, cols, weights_on_grid, b);
#pragma unroll
        for (int k = 0; k < P; ++k) f[i][k] = fma2(mul2(f[i][k], scale), w[k], b[k]);
      } else {
#pragma unroll
        for (int k = 0; k < P; ++k) f[i][k] = mul2(mul2(f[i][k], scale), w[k]);
      }
      uint32_t o[4];
      pack2<DT, P>(f[i], o);
      units.store(static_cast<char*>(a.out[r]) + at, u, o);
    }
    if (t == 0 && a.mean[r] != nullptr) {
      a.mean[r][row] = mean;
      a.rstd[r][row] = rstd;
    }
  }
}

// ------------------------------------------------------------------- backward
// What a unit of x and dy adds to a row's two sums and to the sums over rows.
template <int DT, int P>
__device__ __forceinline__ void add_unit(const uint4& xv, const uint4& dv, const F2* weight, F2 rstd, F2 shift, F2& sg, F2& sgz, F2* dw, F2* db) {
  const uint32_t x[4] = {xv.x, xv.y, xv.z, xv.w}, dy[4] = {dv.x, dv.y, dv.z, dv.w};
#pragma unroll
  for (int k = 0; k < P; ++k) {
    const F2 z = fma2(widen2<DT>(x, k), rstd, shift), d = widen2<DT>(dy, k), g = mul2(d, weight[k]);
    sg = add2(sg, g);
    sgz = fma2(g, z, sgz);
    dw[k] = fma2(d, z, dw[k]);
    db[k] = add2(db[k], d);
  }
}
// dx of a unit; means: -mean(g) and -mean(g z).
template <int DT, int P, bool EXTRA>
__device__ __forceinline__ void grad_unit(const uint4& xv, const uint4& dv, const uint4& ev, const F2* weight, F2 rstd, F2 shift, F2 mean_g, F2 mean_gz,
                                          uint32_t* o) {
  const uint32_t x[4] = {xv.x, xv.y, xv.z, xv.w}, dy[4] = {dv.x, dv.y, dv.z, dv.w}, more[4] = {ev.x, ev.y, ev.z, ev.w};
  F2 f[P];
#pragma unroll
  for (int k = 0; k < P; ++k) {
    const F2 z = fma2(widen2<DT>(x, k), rstd, shift);
    f[k] = fma2(z, mean_gz, fma2(widen2<DT>(dy, k), weight[k], mean_g));
    f[k] = EXTRA ? fma2(f[k], rstd, widen2<DT>(more, k)) : mul2(f[k], rstd);
  }
  pack2<DT, P>(f, o);
}

// The sums over rows of a CTA's groups, group after group, to its part.
template <int VEC, int U>
__device__ __forceinline__ void write_part(const NormArgs& a, const Group& group, int groups, int group_threads, float* shared,
                                           const F2 (&dw)[U][VEC / 2], const F2 (&db)[U][VEC / 2]) {
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
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const uint32_t c = (t + i * group_threads) * VEC + e;
        if (c >= cols) break;
        const float2 w = parts(dw[i][e / 2]), b = parts(db[i][e / 2]);
        const float vw = e & 1 ? w.y : w.x, vb = e & 1 ? b.y : b.x;
        to[c] = g == 0 ? vw : shared[c] + vw;
        to[cols + c] = g == 0 ? vb : shared[cols + c] + vb;
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
  constexpr int VEC = 16 / Elem<DT>::kBytes, P = VEC / 2, ARRAYS = EXTRA ? 3 : 2, PER_STAGE = R * ARRAYS * U;
  extern __shared__ uint4 ring[];  // [depth][R][ARRAYS][U][threads]
  __shared__ float4 slots[2 * kMostWarps];
  pdl_enter();
  Group group(slots, group_threads);
  const RowPart part = row_part(a.parts, a.p, blockIdx.x);
  const int r = part.r, groups = blockDim.x / group_threads, t = threadIdx.x - group.id * group_threads;
  const uint32_t cols = a.cols, units = cols / VEC;
  const uint64_t row_bytes = static_cast<uint64_t>(cols) * Elem<DT>::kBytes;
  const float inv = 1.f / static_cast<float>(cols);
  const uint4* mine = ring + threadIdx.x;
  const uint32_t mine_at = static_cast<uint32_t>(__cvta_generic_to_shared(mine)), step = blockDim.x * 16;
  F2 dw[U][P], db[U][P];
#pragma unroll
  for (int i = 0; i < U; ++i)
#pragma unroll
    for (int k = 0; k < P; ++k) dw[i][k] = db[i][k] = both(0.f);

  const char *x = static_cast<const char*>(a.x[r]) + t * 16, *dy = static_cast<const char*>(a.dy[r]) + t * 16;
  const char* extra = static_cast<const char*>(a.extra[r]) + t * 16;
  char* out = static_cast<char*>(a.out[r]) + t * 16;
  const uint32_t hop = group_threads * 16;
  const auto fetch = [&](uint64_t row0, int stage) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (row0 + j >= part.hi) break;
      const uint64_t at = (row0 + j) * row_bytes;
      const uint32_t to = mine_at + (stage * PER_STAGE + j * ARRAYS * U) * step;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (t + i * group_threads >= units) break;
        copy16_async(to + i * step, x + at + i * hop);
        copy16_async(to + (U + i) * step, dy + at + i * hop);
        if constexpr (EXTRA) copy16_async(to + (2 * U + i) * step, extra + at + i * hop);
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
      const int next = stage + depth - 1;
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
    F2 sg[R], sgz[R];
#pragma unroll
    for (int j = 0; j < R; ++j) sg[j] = sgz[j] = both(0.f);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t u = t + i * group_threads;
      if (u >= units) break;
      F2 weight[P];
      load_weights<WT, VEC>(a.weight[r], u * VEC, cols, weights_on_grid, weight);
#pragma unroll
      for (int j = 0; j < R; ++j) {
        if (row0 + j >= part.hi) break;
        add_unit<DT, P>(here[(j * ARRAYS * U + i) * blockDim.x], here[(j * ARRAYS * U + U + i) * blockDim.x], weight, both(rstd[j]),
                        both(-mean[j] * rstd[j]), sg[j], sgz[j], dw[i], db[i]);
      }
    }
    float sums[2 * R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      sums[2 * j] = total2(sg[j]);
      sums[2 * j + 1] = total2(sgz[j]);
    }
    group.sum<2 * R>(sums);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t u = t + i * group_threads;
      if (u >= units) break;
      F2 weight[P];
      load_weights<WT, VEC>(a.weight[r], u * VEC, cols, weights_on_grid, weight);
#pragma unroll
      for (int j = 0; j < R; ++j) {
        if (row0 + j >= part.hi) break;
        uint4 more = make_uint4(0, 0, 0, 0);
        if constexpr (EXTRA) more = here[(j * ARRAYS * U + 2 * U + i) * blockDim.x];
        uint32_t o[4];
        grad_unit<DT, P, EXTRA>(here[(j * ARRAYS * U + i) * blockDim.x], here[(j * ARRAYS * U + U + i) * blockDim.x], more, weight, both(rstd[j]),
                                both(-mean[j] * rstd[j]), both(-sums[2 * j] * inv), both(-sums[2 * j + 1] * inv), o);
        st_stream16(out + (row0 + j) * row_bytes + i * hop, make_uint4(o[0], o[1], o[2], o[3]));
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

// Rows off the grid, or too long for a ring: a row waits in registers, the next one
// is on its way there.
template <int DT, int WT, int U, bool EXTRA>
__global__ void __launch_bounds__(512) norm_grad_off_kernel(const __grid_constant__ NormArgs a, int group_threads, uint32_t weights_on_grid) {
  constexpr int VEC = 16 / Elem<DT>::kBytes, P = VEC / 2;
  extern __shared__ uint4 ring[];
  __shared__ float4 slots[2 * kMostWarps];
  pdl_enter();
  Group group(slots, group_threads);
  const RowPart part = row_part(a.parts, a.p, blockIdx.x);
  const int r = part.r, groups = blockDim.x / group_threads, t = threadIdx.x - group.id * group_threads;
  const uint32_t cols = a.cols;
  const Units<DT, false> units(cols);
  const float inv = 1.f / static_cast<float>(cols);
  const char *x = static_cast<const char*>(a.x[r]), *dy = static_cast<const char*>(a.dy[r]), *extra = static_cast<const char*>(a.extra[r]);
  F2 dw[U][P], db[U][P];
#pragma unroll
  for (int i = 0; i < U; ++i)
#pragma unroll
    for (int k = 0; k < P; ++k) dw[i][k] = db[i][k] = both(0.f);
  uint64_t row = part.lo + static_cast<uint64_t>(group.id);
  uint4 next_x[U], next_dy[U];
  float next_mean = 0.f, next_rstd = 0.f;
  const auto fetch = [&](uint64_t row) {
    if (row >= part.hi) return;
    const uint64_t at = row * units.row_bytes;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      next_x[i] = units.load(x + at, t + i * group_threads);
      next_dy[i] = units.load(dy + at, t + i * group_threads);
    }
    next_mean = a.mean[r][row];
    next_rstd = a.rstd[r][row];
  };
  fetch(row);
  for (; row < part.hi; row += groups) {
    uint4 xv[U], dv[U], ev[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      xv[i] = next_x[i];
      dv[i] = next_dy[i];
    }
    const F2 rstd = both(next_rstd), shift = both(-next_mean * next_rstd);
    const uint64_t at = row * units.row_bytes;
    if constexpr (EXTRA) {
#pragma unroll
      for (int i = 0; i < U; ++i) ev[i] = units.load(extra + at, t + i * group_threads);
    }
    fetch(row + groups);
    F2 sg = both(0.f), sgz = both(0.f);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t u = t + i * group_threads;
      if (u >= units.count) break;
      F2 weight[P];
      load_weights<WT, VEC>(a.weight[r], u * VEC, cols, weights_on_grid, weight);
      add_unit<DT, P>(xv[i], dv[i], weight, rstd, shift, sg, sgz, dw[i], db[i]);
    }
    float sums[2] = {total2(sg), total2(sgz)};
    group.sum<2>(sums);
    const F2 mean_g = both(-sums[0] * inv), mean_gz = both(-sums[1] * inv);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t u = t + i * group_threads;
      F2 weight[P];
      load_weights<WT, VEC>(a.weight[r], u * VEC, cols, weights_on_grid, weight);
      uint32_t o[4];
      grad_unit<DT, P, EXTRA>(xv[i], dv[i], ev[i], weight, rstd, shift, mean_g, mean_gz, o);
      units.store(static_cast<char*>(a.out[r]) + at, u, o);
    }
  }
  write_part<VEC, U>(a, group, groups, group_threads, reinterpret_cast<float*>(ring), dw, db);
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
    const uint32_t units = (a.cols * Elem<DT>::kBytes + 15) / 16;
    const auto go = [&](auto un) {
      constexpr int U = decltype(un)::value;
      const int group = whole_warps(units, U), groups = group >= 256 ? 1 : 256 / group;
      // parts small enough that the last ones of a launch end together
      cut_rows(&a.parts, rows, a.p, 152 * 32, groups, false);
      return launch_norm_kernel(vec ? (sum ? norm_kernel<DT, WT, U, true, true> : norm_kernel<DT, WT, U, false, true>)
                                    : (sum ? norm_kernel<DT, WT, U, true, false> : norm_kernel<DT, WT, U, false, false>),
                                a.parts.first[a.p], group * groups, 0, s, a, group, grid);
    };
    if (units <= 32) return go(Int<1>{});
    if (units <= 64) return go(Int<2>{});
    return units <= 2048 ? go(Int<4>{}) : go(Int<8>{});
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
      const int group = whole_warps((a.cols + VEC - 1) / VEC, U), groups = group >= 256 ? 1 : 256 / group;
      return launch(extra ? norm_grad_off_kernel<DT, WT, U, true> : norm_grad_off_kernel<DT, WT, U, false>, kNormParts, group, groups, 1,
                    groups > 1 ? a.cols * 8 : 0, grid);
    };
    const auto any_off = [&] {
      if (a.cols <= 256) return off(Int<8 / VEC>{});
      return a.cols <= 8192 ? off(Int<16 / VEC>{}) : off(Int<32 / VEC>{});
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
