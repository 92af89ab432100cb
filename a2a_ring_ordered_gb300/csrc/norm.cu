// norm.cu -- layer norm over rows, and its gradients.
//
//   v = x (+ residual, rounded to the rows' type), m = mean(v),
//   s = (mean((v - m)^2) + eps)^-1/2,  y = (v - m) s w + b;
//   with z = (v - m) s and g = dy w:
//   dx = s (g - mean(g) - z mean(g z)) + dsum,  dw = sum over rows of dy z,  db = of dy.
//
// Rows move once in each direction, so HBM bounds all of it, where enough loads are
// under way.  A group of one or more warps has a row, which stays in registers
// between the walks over it; a thread has the same columns of every row that its
// group takes, so that the sums over rows stay in its registers too, or in its own
// slots of shared memory.
// Measured, of 8 ranks x 4096 rows of 7168 bf16 with fp32 weights and a residual:
// forward 301 us (6.2 TB/s), gradients 300 (6.25); without a residual, 34,877 rows,
// 214 us (4.7) and 267 (5.6); 14,006 fp32 rows of 1019, off the grid, 22 us (5.1),
// gradients of 25,998 bf16 ones 42 us (3.8).
#include "pairs.cuh"
#include "row_parts.cuh"

namespace ccl {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;

// ------------------------------------------------------------------- units
// On the grid (all rows start on 16 bytes and are multiples of them) a row goes in
// units of 16 bytes, off it in elements; thread t of a group has units t, t +
// threads, ...: the same columns in every row.

// The row's granules into L2, by one instruction: a group asks for its next row
// while it works on one.
__device__ __forceinline__ void prefetch_row(const void* base, uint64_t at, uint32_t row_bytes) {
  const uintptr_t start = reinterpret_cast<uintptr_t>(base) + at, granule = start & ~static_cast<uintptr_t>(15);
  const uint32_t size = static_cast<uint32_t>((start + row_bytes - granule + 15) & ~static_cast<uintptr_t>(15));
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(granule), "r"(size) : "memory");
}

// The vectors of a call: weight or bias, of fp32 or bf16.
struct Vector {
  const void* base;
  int dt;
  bool grid;  // starts on 16 bytes
};
// The N (4 or 8) columns from c on, a multiple of N.
template <int N>
__device__ __forceinline__ void load_columns(const Vector& v, uint32_t c, F2* f) {
  if (v.dt == kF32) {
    const float* p = static_cast<const float*>(v.base) + c;
#pragma unroll
    for (int k = 0; k < N / 4; ++k) {
      const float4 q = v.grid ? reinterpret_cast<const float4*>(p)[k] : make_float4(p[4 * k], p[4 * k + 1], p[4 * k + 2], p[4 * k + 3]);
      f[2 * k] = pair(q.x, q.y);
      f[2 * k + 1] = pair(q.z, q.w);
    }
  } else {
    const unsigned short* p = static_cast<const unsigned short*>(v.base) + c;
    uint32_t w[N / 2];
    if (v.grid) {
#pragma unroll
      for (int k = 0; k < N / 4; ++k) {
        const uint2 q = reinterpret_cast<const uint2*>(p)[k];
        w[2 * k] = q.x;
        w[2 * k + 1] = q.y;
      }
    } else {
#pragma unroll
      for (int k = 0; k < N / 2; ++k) w[k] = p[2 * k] | static_cast<uint32_t>(p[2 * k + 1]) << 16;
    }
#pragma unroll
    for (int k = 0; k < N / 2; ++k) f[k] = widen2<kBF16>(w, k);
  }
}
// The same from shared memory, where a vector lies in planes of every unit's first,
// second, ... four columns: the lanes' 16 bytes are neighbours.
template <int N>
__device__ __forceinline__ void staged_columns(const float4* planes, uint32_t units, uint32_t u, F2* f) {
#pragma unroll
  for (int k = 0; k < N / 4; ++k) {
    const float4 q = planes[k * units + u];
    f[2 * k] = pair(q.x, q.y);
    f[2 * k + 1] = pair(q.z, q.w);
  }
}
template <int N>
__device__ __forceinline__ void stage_columns(const Vector& v, float4* planes, uint32_t units) {
  for (uint32_t u = threadIdx.x; u < units; u += blockDim.x) {
    F2 f[N / 2];
    load_columns<N>(v, u * N, f);
#pragma unroll
    for (int k = 0; k < N / 4; ++k) {
      const float2 a = parts(f[2 * k]), b = parts(f[2 * k + 1]);
      planes[k * units + u] = make_float4(a.x, a.y, b.x, b.y);
    }
  }
}

// Off the grid: how many columns thread t of G has, and its columns of a row, two
// to a pair, from the first one's place on; zeros behind them.
template <int G>
__device__ __forceinline__ int own_columns(uint32_t cols, int t) {
  return static_cast<int>(cols / G) + (t < static_cast<int>(cols % G) ? 1 : 0);
}
// Of U, as many as every thread has by the choice of G and U (by_columns), which
// need no look at `mine`: 1019 columns of bf16 forward 3.8 -> 4.2 TB/s.
template <int G, int U>
constexpr int kSure = G >= 64 ? U / 2 : U >= 16 ? U / 4 : 0;
template <int DT, int G, int U>
__device__ __forceinline__ void load_row(const char* at, int mine, F2* f) {
  float v[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    v[i] = 0.f;
    if (i < kSure<G, U> || i < mine) {
      if constexpr (DT == kF32) v[i] = reinterpret_cast<const float*>(at)[i * G];
      else v[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(at)[i * G]);
    }
  }
#pragma unroll
  for (int k = 0; k < U / 2; ++k) f[k] = pair(v[2 * k], v[2 * k + 1]);
}
// The same in two steps: the elements' bits, and the columns of these.
template <int DT, int G, int U>
__device__ __forceinline__ void load_bits(const char* at, int mine, uint32_t* v) {
#pragma unroll
  for (int i = 0; i < U; ++i) {
    v[i] = 0;
    if (i < kSure<G, U> || i < mine) {
      if constexpr (DT == kF32) v[i] = reinterpret_cast<const uint32_t*>(at)[i * G];
      else v[i] = reinterpret_cast<const unsigned short*>(at)[i * G];
    }
  }
}
template <int DT, int U>
__device__ __forceinline__ void floats_of(const uint32_t* v, F2* f) {
  constexpr int kShift = DT == kF32 ? 0 : 16;
#pragma unroll
  for (int k = 0; k < U / 2; ++k) f[k] = pair(__uint_as_float(v[2 * k] << kShift), __uint_as_float(v[2 * k + 1] << kShift));
}
template <int G, int U>
__device__ __forceinline__ void load_spread(const void* base, int dt, int t, int mine, F2* f) {
  if (dt == kF32) load_row<kF32, G, U>(static_cast<const char*>(base) + t * 4, mine, f);
  else load_row<kBF16, G, U>(static_cast<const char*>(base) + t * 2, mine, f);
}
template <int DT, int U>
__device__ __forceinline__ void round_row(F2* f) {
  if constexpr (DT == kBF16) {
#pragma unroll
    for (int k = 0; k < U / 2; ++k) {
      uint32_t o;
      pack2<DT, 1>(f + k, &o);
      f[k] = widen2<DT>(&o, 0);
    }
  }
}
template <int DT, int G, int U>
__device__ __forceinline__ void store_row(char* at, int mine, const F2* f) {
#pragma unroll
  for (int k = 0; k < U / 2; ++k) {
    uint32_t o[2];
    pack2<DT, 1>(f + k, o);
    if (2 * k < kSure<G, U> || 2 * k < mine) store_one<DT>(at, 2 * k * G, o, 0);
    if (2 * k + 1 < kSure<G, U> || 2 * k + 1 < mine) store_one<DT>(at, (2 * k + 1) * G, o, 1);
  }
}

// ------------------------------------------------------------ groups of warps
// One or two sums over a group, the same for every thread and in a fixed order:
// by shuffles within the warps, then through shared memory in two sets of slots
// in turn, so that one barrier of the group does for each sum.  Two sums share
// their shuffles: the lower half of the lanes takes the one, the upper half the
// other.
constexpr int kMostWarps = 16;   // of a group
constexpr int kMostGroups = 8;   // of a CTA, that have more than a warp
struct Group {
  int warps, warp, lane, id;  // warps of the group, this one among them, the group's number
  int turn = 0;
  float* slots;               // [2][kMostGroups][2 * kMostWarps]; zeros where there is no warp
  __device__ __forceinline__ Group(float (&s)[2][kMostGroups][2 * kMostWarps], int group_threads) {
    warps = group_threads >> 5;
    id = static_cast<int>(threadIdx.x) / group_threads;
    warp = (static_cast<int>(threadIdx.x) - id * group_threads) >> 5;
    lane = threadIdx.x & 31;
    if (warps == 1) return;
    slots = s[0][id];
    if (warp < 2) s[warp][id][lane] = 0.f;
    sync();
  }
  __device__ __forceinline__ void sync() const {
    asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(warps * 32) : "memory");
  }
  __device__ __forceinline__ float across(float v) {
    float* s = slots + turn * (kMostGroups * 2 * kMostWarps);
    turn ^= 1;
    if ((lane & 15) == 0) s[lane + warp] = v;
    sync();
    v = s[lane];
#pragma unroll
    for (int o = kMostWarps / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
  }
  __device__ __forceinline__ float2 sum(float a, float b) {
    const bool upper = lane >= 16;
    float v = (upper ? b : a) + __shfl_xor_sync(kAll, upper ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    if (warps > 1) v = across(v);
    return make_float2(__shfl_sync(kAll, v, 0), __shfl_sync(kAll, v, 16));
  }
  __device__ __forceinline__ float sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return warps > 1 ? across(v) : v;
  }
};

// -------------------------------------------------------------------- forward
// The row stays in registers between its three walks (mean, variance, output).
// weight and bias come from shared memory where a CTA has rows enough (`stage`):
// from L1, where a lane's eight fp32 columns lie 32 bytes from its neighbour's, they
// took 80 % of its bandwidth and 252 us for 34,877 rows of 7168 bf16, 214 so.
template <int DT, int U, bool SUM>
__global__ void __maxnreg__(U * 16 / Elem<DT>::kBytes <= 16 ? 64 : U * 16 / Elem<DT>::kBytes <= 32 ? 80 : 128) norm_kernel(const __grid_constant__ NormArgs a, int group_threads, int weight_dt, uint32_t weights_on_grid, int stage) {
  constexpr int VEC = 16 / Elem<DT>::kBytes, P = VEC / 2;
  extern __shared__ float4 planes[];  // stage: the weight's VEC / 4 planes, then the bias's
  __shared__ float slots[2][kMostGroups][2 * kMostWarps];
  pdl_enter();
  Group group(slots, group_threads);
  const RowPart part = row_part(a.parts, a.p, blockIdx.x);
  const int r = part.r, groups = blockDim.x / group_threads, t = threadIdx.x - group.id * group_threads;
  const uint32_t cols = a.cols, units = cols / VEC, row_bytes = cols * Elem<DT>::kBytes;
  const Vector weight{a.weight[r], weight_dt, weights_on_grid != 0}, bias{a.bias[r], weight_dt, weights_on_grid != 0};
  float4* const bias_planes = planes + units * (VEC / 4);
  if (stage) {
    stage_columns<VEC>(weight, planes, units);
    if (bias.base != nullptr) stage_columns<VEC>(bias, bias_planes, units);
    __syncthreads();
  }
  const float n = static_cast<float>(cols), eps = static_cast<float>(a.eps);
  for (uint32_t row = part.lo + group.id; row < part.hi; row += groups) {
    const uint64_t at = static_cast<uint64_t>(row) * row_bytes;
    if (t == 0 && part.hi - row > static_cast<uint32_t>(groups)) {
      prefetch_row(a.x[r], at + static_cast<uint64_t>(groups) * row_bytes, row_bytes);
      if constexpr (SUM) prefetch_row(a.extra[r], at + static_cast<uint64_t>(groups) * row_bytes, row_bytes);
    }
    F2 f[U][P];
    {
      uint4 v[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const uint32_t u = t + i * group_threads;
        v[i] = u < units ? ld_once16(static_cast<const char*>(a.x[r]) + at + 16 * u) : make_uint4(0, 0, 0, 0);
      }
      if constexpr (SUM) {
        uint4 q[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const uint32_t u = t + i * group_threads;
          q[i] = u < units ? ld_once16(static_cast<const char*>(a.extra[r]) + at + 16 * u) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const uint32_t u = t + i * group_threads;
          uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w}, o[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
          if constexpr (DT == kBF16) {
            // the sum of two bf16 numbers rounded to bf16 at once, or by way of fp32, is the same
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __nv_bfloat162 h = __hadd2(*reinterpret_cast<__nv_bfloat162*>(&w[k]), *reinterpret_cast<__nv_bfloat162*>(&o[k]));
              w[k] = *reinterpret_cast<const uint32_t*>(&h);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = __float_as_uint(__uint_as_float(w[k]) + __uint_as_float(o[k]));
          }
          v[i] = make_uint4(w[0], w[1], w[2], w[3]);
          if (u < units) st_stream16(static_cast<char*>(a.sum[r]) + at + 16 * u, v[i]);
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
    const float mean = group.sum(total2(sum)) / n;
    const F2 less = both(-mean);
    sum = both(0.f);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (t + i * group_threads >= units) break;
#pragma unroll
      for (int k = 0; k < P; ++k) {
        f[i][k] = add2(f[i][k], less);
        sum = fma2(f[i][k], f[i][k], sum);
      }
    }
    const float rstd = 1.f / sqrtf(group.sum(total2(sum)) / n + eps);
    const F2 scale = both(rstd);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t u = t + i * group_threads;
      if (u >= units) break;
      F2 w[P], b[P];
      if (stage) staged_columns<VEC>(planes, units, u, w);
      else load_columns<VEC>(weight, u * VEC, w);
      if (bias.base != nullptr) {
        if (stage) staged_columns<VEC>(bias_planes, units, u, b);
        else load_columns<VEC>(bias, u * VEC, b);
#pragma unroll
        for (int k = 0; k < P; ++k) f[i][k] = fma2(mul2(f[i][k], scale), w[k], b[k]);
      } else {
#pragma unroll
        for (int k = 0; k < P; ++k) f[i][k] = mul2(mul2(f[i][k], scale), w[k]);
      }
      uint32_t o[4];
      pack2<DT, P>(f[i], o);
      st_stream16(static_cast<char*>(a.out[r]) + at + 16 * u, make_uint4(o[0], o[1], o[2], o[3]));
    }
    if (t == 0 && a.mean[r] != nullptr) {
      a.mean[r][row] = mean;
      a.rstd[r][row] = rstd;
    }
  }
}

// Rows off the grid, by elements: thread t of G has columns t + G i, and their
// weights in registers too.
template <int DT, int G, int U, bool SUM>
__global__ void __launch_bounds__(G > 256 ? G : 256, G > 256 ? 1 : 3) norm_off_kernel(const __grid_constant__ NormArgs a, int weight_dt) {
  constexpr int B = Elem<DT>::kBytes, H = U / 2;
  __shared__ float slots[2][kMostGroups][2 * kMostWarps];
  pdl_enter();
  Group group(slots, G);
  const RowPart part = row_part(a.parts, a.p, blockIdx.x);
  const int r = part.r, groups = blockDim.x / G, t = threadIdx.x % G;
  const uint32_t cols = a.cols, row_bytes = cols * B;
  const int mine = own_columns<G>(cols, t);
  const float n = static_cast<float>(cols), eps = static_cast<float>(a.eps);
  F2 w[H], b[H];
  load_spread<G, U>(a.weight[r], weight_dt, t, mine, w);
  if (a.bias[r] != nullptr) {
    load_spread<G, U>(a.bias[r], weight_dt, t, mine, b);
  } else {
#pragma unroll
    for (int k = 0; k < H; ++k) b[k] = both(0.f);
  }
  for (uint32_t row = part.lo + group.id; row < part.hi; row += groups) {
    const uint64_t at = static_cast<uint64_t>(row) * row_bytes;
    if (t == 0 && part.hi - row > static_cast<uint32_t>(groups)) {
      prefetch_row(a.x[r], at + static_cast<uint64_t>(groups) * row_bytes, row_bytes);
      if constexpr (SUM) prefetch_row(a.extra[r], at + static_cast<uint64_t>(groups) * row_bytes, row_bytes);
    }
    F2 f[H];
    load_row<DT, G, U>(static_cast<const char*>(a.x[r]) + at + t * B, mine, f);
    if constexpr (SUM) {
      F2 q[H];
      load_row<DT, G, U>(static_cast<const char*>(a.extra[r]) + at + t * B, mine, q);
#pragma unroll
      for (int k = 0; k < H; ++k) f[k] = add2(f[k], q[k]);
      round_row<DT, U>(f);
      store_row<DT, G, U>(static_cast<char*>(a.sum[r]) + at + t * B, mine, f);
    }
    F2 sum = both(0.f);
#pragma unroll
    for (int k = 0; k < H; ++k) sum = add2(sum, f[k]);
    const float mean = group.sum(total2(sum)) / n;
    const F2 less = both(-mean);
    sum = both(0.f);
#pragma unroll
    for (int k = 0; k < H; ++k) {
      f[k] = add2(f[k], less);
      if (2 * k + 2 > mine) f[k] = pair(2 * k < mine ? parts(f[k]).x : 0.f, 0.f);
      sum = fma2(f[k], f[k], sum);
    }
    const float rstd = 1.f / sqrtf(group.sum(total2(sum)) / n + eps);
    const F2 scale = both(rstd);
#pragma unroll
    for (int k = 0; k < H; ++k) f[k] = fma2(mul2(f[k], scale), w[k], b[k]);
    store_row<DT, G, U>(static_cast<char*>(a.out[r]) + at + t * B, mine, f);
    if (t == 0 && a.mean[r] != nullptr) {
      a.mean[r][row] = mean;
      a.rstd[r][row] = rstd;
    }
  }
}

// ------------------------------------------------------------------- backward
template <int N>
__device__ __forceinline__ void spread2(const F2* f, float* v) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const float2 t = parts(f[k]);
    v[2 * k] = t.x;
    v[2 * k + 1] = t.y;
  }
}

// z is (x - mean) rstd, as in the forward pass: by one fused multiply-add with a
// rounded mean rstd it would be off by 2^-24 of that, however small itself (this
// costs 7168 bf16 columns 1.6 %, 248.5 -> 252.5 us for 32,768 rows).  rstd for z:
// where mean rstd is beyond fp32, the row's elements are its mean (one that is not
// differs by 2^-24 of it at least, and the row deviates accordingly), so z is 0;
// rstd would make infinities of the zeros behind the row.
__device__ __forceinline__ float z_scale(float mean, float rstd) {
  return isinf(mean * rstd) && !isinf(rstd) ? 0.f : rstd;
}

// The sums over rows of a CTA's groups, group after group, to its part.
template <int VEC, int U>
__device__ __forceinline__ void write_part(const NormArgs& a, const Group& group, int groups, int group_threads, float* shared,
                                           const float* dw, const float* db) {
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
        const float vw = dw[i * VEC + e], vb = db[i * VEC + e];
        to[c] = g == 0 ? vw : shared[c] + vw;
        to[cols + c] = g == 0 ? vb : shared[cols + c] + vb;
      }
  }
}

// The sums over rows where registers do not hold them beside z and g (32 columns a
// thread), or are wanted for other things: four columns to a slot, a thread's own, in
// planes over the threads.  Only where a CTA is one group.  12,288 columns of bf16 go
// at 4.2 TB/s so (5.5 with dsum), 10,001 at 2.65; spilled by the compiler, at 3.4 (4.05)
// and 1.15.
template <int Q>
struct SharedSums {
  float4 *w, *b;
  int threads;
  __device__ __forceinline__ SharedSums(float* shared, int group_threads, int t)
      : w(reinterpret_cast<float4*>(shared) + t), b(w + Q * group_threads), threads(group_threads) {}
  __device__ __forceinline__ void clear() const {
#pragma unroll
    for (int q = 0; q < Q; ++q) w[q * threads] = b[q * threads] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void add(int q, F2 d0, F2 d1, F2 z0, F2 z1) const {
    const float4 sw = w[q * threads], sb = b[q * threads];
    const float2 w0 = parts(fma2(d0, z0, pair(sw.x, sw.y))), w1 = parts(fma2(d1, z1, pair(sw.z, sw.w)));
    const float2 b0 = parts(add2(d0, pair(sb.x, sb.y))), b1 = parts(add2(d1, pair(sb.z, sb.w)));
    w[q * threads] = make_float4(w0.x, w0.y, w1.x, w1.y);
    b[q * threads] = make_float4(b0.x, b0.y, b1.x, b1.y);
  }
  __device__ __forceinline__ void get(float* all_w, float* all_b) const {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const float4 sw = w[q * threads], sb = b[q * threads];
      all_w[4 * q] = sw.x, all_w[4 * q + 1] = sw.y, all_w[4 * q + 2] = sw.z, all_w[4 * q + 3] = sw.w;
      all_b[4 * q] = sb.x, all_b[4 * q + 1] = sb.y, all_b[4 * q + 2] = sb.z, all_b[4 * q + 3] = sb.w;
    }
  }
};

// Rows on the 16-byte grid.  z and g stay in registers between the row's two walks;
// with PRE the next row's units are on the way to registers meanwhile, and the
// row after it to L2, else the next row to L2; HELD: the sums over rows are in
// registers.  The bounds name the threads that a
// width takes: the compiler's order of the same instructions for 512 threads cost 15 %
// at 448.  For 8 x 4096 rows of 7168 bf16 with dsum, 300 us so, a ring of asynchronous
// copies three rows deep took 410, the second walk from L1 and two rows a SM 447, half
// the columns a thread 445 (all before the two steps above: 352 us).
template <int DT, int U, bool EXTRA, bool PRE, bool HELD, int MOST, int PER_SM>
__global__ void __launch_bounds__(MOST, PER_SM) norm_grad_kernel(const __grid_constant__ NormArgs a, int group_threads, int weight_dt, uint32_t weights_on_grid) {
  constexpr int VEC = 16 / Elem<DT>::kBytes, P = VEC / 2;
  constexpr bool LATE = U * VEC > 8;  // dsum after the first walk, for its registers' sake: 352 -> 323 us
  extern __shared__ float shared[];
  __shared__ float slots[2][kMostGroups][2 * kMostWarps];
  pdl_enter();
  Group group(slots, group_threads);
  const RowPart part = row_part(a.parts, a.p, blockIdx.x);
  const int r = part.r, groups = blockDim.x / group_threads, t = threadIdx.x - group.id * group_threads;
  const uint32_t cols = a.cols, row_bytes = cols * Elem<DT>::kBytes, hop = group_threads * 16;
  const int mine = (static_cast<int>(cols / VEC) - t + group_threads - 1) / group_threads;  // units of the thread
  const float inv = 1.f / static_cast<float>(cols);
  const Vector weight{a.weight[r], weight_dt, weights_on_grid != 0};
  F2 dw[HELD ? U : 1][P], db[HELD ? U : 1][P];
  const SharedSums<U * VEC / 4> away(shared, group_threads, t);
  if constexpr (HELD) {
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int k = 0; k < P; ++k) dw[i][k] = db[i][k] = both(0.f);
  } else {
    away.clear();
  }
  uint4 x[U], dy[U], extra[U];
  const auto load = [&](const void* from, uint32_t row, uint4* to) {
    const char* at = static_cast<const char*>(from) + static_cast<uint64_t>(row) * row_bytes + t * 16;
#pragma unroll
    for (int i = 0; i < U; ++i) to[i] = i < mine ? ld_once16(at + i * hop) : make_uint4(0, 0, 0, 0);
  };
  // rows are below 2^31, groups few
  uint32_t row = part.lo + group.id;
  float mean = 0.f, rstd = 0.f;
  const auto fetch = [&](uint32_t row) {
    load(a.x[r], row, x);
    load(a.dy[r], row, dy);
    mean = a.mean[r][row];
    rstd = a.rstd[r][row];
  };
  if (PRE && row < part.hi) fetch(row);
  for (; row < part.hi; row += groups) {
    const uint32_t far = row + (PRE ? 2 : 1) * groups, after = row + groups;
    if (t < (EXTRA ? 3 : 2) && far < part.hi)
      prefetch_row(t == 0 ? a.x[r] : t == 1 ? a.dy[r] : a.extra[r], static_cast<uint64_t>(far) * row_bytes, row_bytes);
    if constexpr (!PRE) fetch(row);
    if (EXTRA && !LATE) load(a.extra[r], row, extra);
    const F2 scale = both(rstd), less = both(-mean), scale_z = both(z_scale(mean, rstd));
    F2 z[U][P], g[U][P], sg = both(0.f), sgz = both(0.f);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      F2 w[P];
      if (i < mine) {
        load_columns<VEC>(weight, (t + i * group_threads) * VEC, w);
      } else {
#pragma unroll
        for (int k = 0; k < P; ++k) w[k] = both(0.f);
      }
      const uint32_t xw[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, yw[4] = {dy[i].x, dy[i].y, dy[i].z, dy[i].w};
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const F2 d = widen2<DT>(yw, k);
        z[i][k] = mul2(add2(widen2<DT>(xw, k), less), scale_z);
        if constexpr (HELD) {
          dw[i][k] = fma2(d, z[i][k], dw[i][k]);
          db[i][k] = add2(db[i][k], d);
        } else if (k % 2 == 1) {
          away.add(i * P / 2 + k / 2, widen2<DT>(yw, k - 1), d, z[i][k - 1], z[i][k]);
        }
        g[i][k] = mul2(d, w[k]);
        sg = add2(sg, g[i][k]);
        sgz = fma2(g[i][k], z[i][k], sgz);
      }
    }
    if (PRE && after < part.hi) fetch(after);
    if (EXTRA && LATE) load(a.extra[r], row, extra);
    const float2 sums = group.sum(total2(sg), total2(sgz));
    const F2 mean_g = both(-sums.x * inv), mean_gz = both(-sums.y * inv);
    char* out = static_cast<char*>(a.out[r]) + static_cast<uint64_t>(row) * row_bytes + t * 16;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (i >= mine) break;
      const uint32_t more[4] = {extra[i].x, extra[i].y, extra[i].z, extra[i].w};
#pragma unroll
      for (int k = 0; k < P; ++k) {
        g[i][k] = fma2(z[i][k], mean_gz, add2(g[i][k], mean_g));
        g[i][k] = EXTRA ? fma2(g[i][k], scale, widen2<DT>(more, k)) : mul2(g[i][k], scale);
      }
      uint32_t o[4];
      pack2<DT, P>(g[i], o);
      st_stream16(out + i * hop, make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
  float all_w[U * VEC], all_b[U * VEC];
  if constexpr (HELD) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      spread2<P>(dw[i], all_w + i * VEC);
      spread2<P>(db[i], all_b + i * VEC);
    }
  } else {
    away.get(all_w, all_b);
  }
  write_part<VEC, U>(a, group, groups, group_threads, shared, all_w, all_b);
}

// Rows off the grid, by elements (thread t of G has columns t + G i): the row stays
// in registers between its two walks.  With PRE the next row's elements are on the way
// to registers meanwhile and the weights are in shared memory, to make room: 25,998
// bf16 rows of 1019 take 42 us so, 47 with the weights in registers.  dsum needs the room
// itself (4.2 TB/s with PRE, 5.3 without), and fp32 rows of more than a warp lose up
// to 6 % with PRE.
template <int DT, int G, int U, bool EXTRA, bool PRE>
__global__ void __launch_bounds__(G > 256 ? G : 256, G > 256 || U > 16 ? 1 : 2) norm_grad_off_kernel(const __grid_constant__ NormArgs a, int, int weight_dt) {
  constexpr int B = Elem<DT>::kBytes, H = U / 2;
  extern __shared__ float shared[];
  __shared__ float slots[2][kMostGroups][2 * kMostWarps];
  pdl_enter();
  Group group(slots, G);
  const RowPart part = row_part(a.parts, a.p, blockIdx.x);
  const int r = part.r, groups = blockDim.x / G, t = threadIdx.x % G;
  const uint32_t cols = a.cols, row_bytes = cols * B;
  const int mine = own_columns<G>(cols, t);
  const float inv = 1.f / static_cast<float>(cols);
  constexpr bool HELD = U <= 16, STAGED = PRE || !HELD;
  F2 dw[HELD ? H : 1], db[HELD ? H : 1], weight[STAGED ? 1 : H];
  float* const behind = shared + (!HELD ? 2 * U * G : groups > 1 ? 2 * cols : 0);
  float2* const staged = reinterpret_cast<float2*>(behind);
  const SharedSums<U / 4> away(shared, G, t);
  if constexpr (HELD) {
#pragma unroll
    for (int k = 0; k < H; ++k) dw[k] = db[k] = both(0.f);
  } else {
    away.clear();
  }
  if constexpr (STAGED) {
    if (group.id == 0) {
      F2 f[H];
      load_spread<G, U>(a.weight[r], weight_dt, t, mine, f);
#pragma unroll
      for (int k = 0; k < H; ++k) staged[k * G + t] = parts(f[k]);
    }
    __syncthreads();
  } else {
    load_spread<G, U>(a.weight[r], weight_dt, t, mine, weight);
  }
  uint32_t row = part.lo + group.id;
  float next_mean = 0.f, next_rstd = 0.f;
  uint32_t next_x[PRE ? U : 1], next_dy[PRE ? U : 1];
  if (row < part.hi) {
    next_mean = a.mean[r][row];
    next_rstd = a.rstd[r][row];
    if constexpr (PRE) {
      const uint64_t at = static_cast<uint64_t>(row) * row_bytes + t * B;
      load_bits<DT, G, U>(static_cast<const char*>(a.x[r]) + at, mine, next_x);
      load_bits<DT, G, U>(static_cast<const char*>(a.dy[r]) + at, mine, next_dy);
    }
  }
  for (; row < part.hi; row += groups) {
    const uint64_t at = static_cast<uint64_t>(row) * row_bytes, hop = static_cast<uint64_t>(groups) * row_bytes;
    const uint32_t left = part.hi - row;
    if (t == 0 && left > static_cast<uint32_t>(groups) * (PRE ? 2 : 1)) {
      const uint64_t next = at + hop * (PRE ? 2 : 1);
      prefetch_row(a.x[r], next, row_bytes);
      prefetch_row(a.dy[r], next, row_bytes);
      if constexpr (EXTRA) prefetch_row(a.extra[r], next, row_bytes);
    }
    F2 z[H], g[H];  // x and dy first
    if constexpr (PRE) {
      floats_of<DT, U>(next_x, z);
      floats_of<DT, U>(next_dy, g);
    } else {
      load_row<DT, G, U>(static_cast<const char*>(a.x[r]) + at + t * B, mine, z);
      load_row<DT, G, U>(static_cast<const char*>(a.dy[r]) + at + t * B, mine, g);
    }
    const F2 rstd = both(next_rstd), less = both(-next_mean), scale_z = both(z_scale(next_mean, next_rstd));
    if (left > static_cast<uint32_t>(groups)) {
      next_mean = a.mean[r][row + groups];
      next_rstd = a.rstd[r][row + groups];
      if constexpr (PRE) {
        load_bits<DT, G, U>(static_cast<const char*>(a.x[r]) + at + hop + t * B, mine, next_x);
        load_bits<DT, G, U>(static_cast<const char*>(a.dy[r]) + at + hop + t * B, mine, next_dy);
      }
    }
    F2 sg = both(0.f), sgz = both(0.f);
#pragma unroll
    for (int k = 0; k < H; ++k) z[k] = mul2(add2(z[k], less), scale_z);
    if constexpr (!HELD) {
#pragma unroll
      for (int k = 0; k < H; k += 2) {
        away.add(k / 2, g[k], g[k + 1], z[k], z[k + 1]);
      }
    }
#pragma unroll
    for (int k = 0; k < H; ++k) {
      if constexpr (HELD) {
        dw[k] = fma2(g[k], z[k], dw[k]);
        db[k] = add2(db[k], g[k]);
      }
      if constexpr (STAGED) {
        const float2 w = staged[k * G + t];
        g[k] = mul2(g[k], pair(w.x, w.y));
      } else {
        g[k] = mul2(g[k], weight[k]);
      }
      sg = add2(sg, g[k]);
      sgz = fma2(g[k], z[k], sgz);
    }
    const float2 sums = group.sum(total2(sg), total2(sgz));
    const F2 mean_g = both(-sums.x * inv), mean_gz = both(-sums.y * inv);
    if constexpr (EXTRA) {
      F2 more[H];
      load_row<DT, G, U>(static_cast<const char*>(a.extra[r]) + at + t * B, mine, more);
#pragma unroll
      for (int k = 0; k < H; ++k) g[k] = fma2(fma2(z[k], mean_gz, add2(g[k], mean_g)), rstd, more[k]);
    } else {
#pragma unroll
      for (int k = 0; k < H; ++k) g[k] = mul2(fma2(z[k], mean_gz, add2(g[k], mean_g)), rstd);
    }
    store_row<DT, G, U>(static_cast<char*>(a.out[r]) + at + t * B, mine, g);
  }
  float all_w[U], all_b[U];
  if constexpr (HELD) {
    spread2<H>(dw, all_w);
    spread2<H>(db, all_b);
  } else {
    away.get(all_w, all_b);
  }
  write_part<1, U>(a, group, groups, G, shared, all_w, all_b);
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

// Calls f(G, U) with the threads a row off the grid gets and the columns that each
// has.
template <typename F>
cudaError_t by_columns(uint32_t cols, F f) {
  if (cols <= 128) return f(Int<32>{}, Int<4>{});
  if (cols <= 512) return f(Int<32>{}, Int<16>{});
  if (cols <= 1024) return f(Int<64>{}, Int<16>{});
  if (cols <= 2048) return f(Int<128>{}, Int<16>{});
  if (cols <= 4096) return f(Int<256>{}, Int<16>{});
  if (cols <= 8192) return f(Int<512>{}, Int<16>{});
  return f(Int<512>{}, Int<32>{});
}

// The numbers of rows, for cutting them anew; whether a rank has one of the buffers.
struct Rows {
  size_t n[kMoeMaxRanks];
  uint64_t total = 0;
  explicit Rows(const NormArgs& a) {
    for (int r = 0; r < a.p; ++r) total += n[r] = a.parts.rows[r];
  }
};
template <typename T>
bool any_of(const T* const* buffers, int p) {
  for (int r = 0; r < p; ++r)
    if (buffers[r] != nullptr) return true;
  return false;
}

}  // namespace

cudaError_t launch_norm(int dt, int weight_dt, bool vec, NormArgs* args, cudaStream_t s) {
  NormArgs& a = *args;
  const Rows rows(a);
  const bool sum = any_of(a.sum, a.p);
  const uint32_t grid = weights_on_grid(a);
  if (!vec) {
    const auto off = [&](auto d) {
      constexpr int DT = decltype(d)::value;
      return by_columns(a.cols, [&](auto gr, auto un) {
        constexpr int G = decltype(gr)::value, U = decltype(un)::value, groups = G >= 256 ? 1 : 256 / G;
        // parts that are all there at once, for their weights' loads: 14,006 fp32 rows of 1019 take 22 us in 3 a SM, 28 in 2 or 4,
        // 41 in 12
        cut_rows(&a.parts, rows.n, a.p, 152 * 3, groups, false);
        return launch_norm_kernel(sum ? norm_off_kernel<DT, G, U, true> : norm_off_kernel<DT, G, U, false>, a.parts.first[a.p], G * groups, 0, s, a, weight_dt);
      });
    };
    return dt == kF32 ? off(Int<kF32>{}) : off(Int<kBF16>{});
  }
  const auto by_type = [&](auto d) {
    constexpr int DT = decltype(d)::value, VEC = 16 / Elem<DT>::kBytes;
    const uint32_t units = a.cols / VEC;
    const auto on = [&](auto un) {
      constexpr int U = decltype(un)::value;
      const int group = whole_warps(units, U), groups = group >= 256 ? 1 : 256 / group;
      auto* kernel = sum ? norm_kernel<DT, U, true> : norm_kernel<DT, U, false>;
      // the ends of a launch cost less with small parts, the weights' way into shared memory with large ones: 8 x 4096 rows of
      // 7168 bf16 with a residual take 303 us in 6 parts a SM, 302 in 12, 298 in 24; 34,877 rows without 206, 214, 227
      cut_rows(&a.parts, rows.n, a.p, 152 * 12, groups, false);
      // worth it from four rows a group on
      const int stage = rows.total >= static_cast<uint64_t>(a.parts.first[a.p]) * groups * 4;
      const size_t smem = stage ? static_cast<size_t>(a.cols) * 4 * (any_of(a.bias, a.p) ? 2 : 1) : 0;
      // the limit belongs to the function, not to the call: always the most that a call may need
      if (smem > 32 * 1024) {  // with what the kernel has besides it stays below the 48 KB that need no leave
        const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kNormMaxCols * 8));
        if (err != cudaSuccess) return err;
      }
      return launch_norm_kernel(kernel, a.parts.first[a.p], group * groups, smem, s, a, group, weight_dt, grid, stage);
    };
    if (units <= 32) return on(Int<1>{});
    if (units <= 64) return on(Int<2>{});
    if constexpr (kNormMaxCols / VEC > 2048) {  // fp32 rows
      if (units > 2048) return on(Int<8>{});
    }
    return on(Int<4>{});
  };
  return dt == kF32 ? by_type(Int<kF32>{}) : by_type(Int<kBF16>{});
}

cudaError_t launch_norm_grad(int dt, int weight_dt, bool vec, NormArgs* args, cudaStream_t s) {
  NormArgs& a = *args;
  const Rows rows(a);
  const bool extra = any_of(a.extra, a.p);
  const uint32_t grid = weights_on_grid(a);
  // groups of a CTA are joined through shared memory: at most 16 KB, as a row of more has a CTA
  const auto launch = [&](auto* kernel, uint32_t ctas, int group, int groups, size_t smem, auto... more) {
    cut_rows(&a.parts, rows.n, a.p, ctas, groups, false);
    if (smem > 32 * 1024) {  // the sums over rows of kNormMaxCols columns, and their weights
      const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kNormMaxCols * 12));
      if (err != cudaSuccess) return err;
    }
    return launch_norm_kernel(kernel, a.parts.first[a.p], group * groups, smem + (groups > 1 ? a.cols * 8 : 0), s, static_cast<const NormArgs&>(a), group, weight_dt, more...);
  };
  if (!vec) {
    const auto off = [&](auto d) {
      constexpr int DT = decltype(d)::value;
      return by_columns(a.cols, [&](auto gr, auto un) {
        constexpr int G = decltype(gr)::value, U = decltype(un)::value, groups = G >= 256 ? 1 : 256 / G;
        constexpr bool PRE = U <= 16 && (DT == kBF16 || G == 32);  // of the kernel without dsum
        const size_t sums = U > 16 ? U * G * 8 : 0, staged = U > 16 || (PRE && !extra) ? U * G * 4 : 0;
        return launch(extra ? norm_grad_off_kernel<DT, G, U, true, false> : norm_grad_off_kernel<DT, G, U, false, PRE>, kNormParts, G, groups, sums + staged);
      });
    };
    return dt == kF32 ? off(Int<kF32>{}) : off(Int<kBF16>{});
  }
  const auto by_type = [&](auto d) {
    constexpr int DT = decltype(d)::value, VEC = 16 / Elem<DT>::kBytes;
    const auto on = [&](auto un, auto pre, auto held, auto mt, auto ps) {
      constexpr int U = decltype(un)::value, MOST = decltype(mt)::value, PER_SM = decltype(ps)::value;
      constexpr bool PRE = decltype(pre)::value != 0, HELD = decltype(held)::value != 0;
      const int group = whole_warps(a.cols / VEC, U), groups = group >= MOST ? 1 : MOST / group;
      return launch(extra ? norm_grad_kernel<DT, U, true, PRE, HELD, MOST, PER_SM> : norm_grad_kernel<DT, U, false, PRE, HELD, MOST, PER_SM>, kNormParts / 2 * PER_SM, group,
                    groups, HELD ? 0 : static_cast<size_t>(group) * U * VEC * 8, grid);
    };
    if (a.cols <= 256) return on(Int<8 / VEC>{}, Int<1>{}, Int<1>{}, Int<256>{}, Int<2>{});
    if (a.cols <= 4096) return on(Int<16 / VEC>{}, Int<1>{}, Int<1>{}, Int<256>{}, Int<2>{});
    // sums in shared memory where that leaves room for a second CTA, or for what is spilled otherwise: gradients of 5120 bf16
    // columns without and with dsum 4.6 and 5.0 TB/s -> 5.0 and 6.1 (fp32 6.45, 6.8 -> 6.1, 5.8), of 7168 fp32 ones 6.1, 5.5 ->
    // 6.25, 6.65 (bf16 5.7, 6.4 -> 4.5, 5.5)
    constexpr bool B = DT == kBF16;
    if (a.cols <= 5120) return on(Int<16 / VEC>{}, Int<1>{}, Int<!B>{}, Int<320>{}, Int<B ? 2 : 1>{});
    if (a.cols <= 7168) return on(Int<16 / VEC>{}, Int<1>{}, Int<B>{}, Int<448>{}, Int<1>{});
    return a.cols <= 8192 ? on(Int<16 / VEC>{}, Int<1>{}, Int<B>{}, Int<512>{}, Int<1>{}) : on(Int<32 / VEC>{}, Int<0>{}, Int<0>{}, Int<512>{}, Int<1>{});
  };
  return dt == kF32 ? by_type(Int<kF32>{}) : by_type(Int<kBF16>{});
}

cudaError_t launch_norm_join(int dw_dt, const NormJoinArgs& a, cudaStream_t s) {
  const dim3 grid((a.cols + 31) / 32, static_cast<unsigned>(a.p));
  const cudaError_t err = dw_dt == kF32 ? launch_kernel(norm_join_kernel<kF32>, grid, dim3(32 * kJoinWarps), s, a)
                                        : launch_kernel(norm_join_kernel<kBF16>, grid, dim3(32 * kJoinWarps), s, a);
  if (err == cudaSuccess) note_launch();
  return err;
}

}  // namespace ccl
