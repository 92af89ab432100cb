// norm.cu -- layer norm over rows, and its gradients.
//
//   v = x (+ residual, rounded to the rows' type), m = mean(v),
//   s = (mean((v - m)^2) + eps)^-1/2,  y = (v - m) s w + b;
//   with z = (v - m) s and g = dy w:
//   dx = s (g - mean(g) - z mean(g z)) + dsum,  dw = sum over rows of dy z,  db = of dy.
#include "row_parts.cuh"

namespace ccl {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;

template <int DT>
__device__ __forceinline__ float load_one(const void* base, uint64_t i) {
  if constexpr (DT == kF32) return static_cast<const float*>(base)[i];
  else return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i]);
}
template <int DT>
__device__ __forceinline__ void save_one(void* base, uint64_t i, float v) {
  if constexpr (DT == kF32) static_cast<float*>(base)[i] = v;
  else static_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(v);
}

// Sums of two values over the CTA, in a fixed order; every thread gets them.
__device__ __forceinline__ float2 cta_sum(float a, float b) {
  __shared__ float2 warp_sum[32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(kAll, a, o);
    b += __shfl_xor_sync(kAll, b, o);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  float2 t = make_float2(0.f, 0.f);
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) {
    t.x += warp_sum[w].x;
    t.y += warp_sum[w].y;
  }
  return t;
}

template <int DT, int WT>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ NormArgs a) {
  pdl_enter();
  const RowPart part = row_part(a.parts, a.p, blockIdx.x);
  const int r = part.r;
  const uint32_t cols = a.cols;
  const float n = static_cast<float>(cols);
  for (uint32_t row = part.lo; row < part.hi; ++row) {
    const uint64_t at = static_cast<uint64_t>(row) * cols;
    const void* v = a.sum[r] != nullptr ? a.sum[r] : a.x[r];
    float s = 0.f;
    for (uint32_t c = threadIdx.x; c < cols; c += kThreads) {
      float x = load_one<DT>(a.x[r], at + c);
      if (a.sum[r] != nullptr) {
        save_one<DT>(a.sum[r], at + c, x + load_one<DT>(a.extra[r], at + c));
        x = load_one<DT>(v, at + c);
      }
      s += x;
    }
    const float mean = cta_sum(s, 0.f).x / n;
    float q = 0.f;
    for (uint32_t c = threadIdx.x; c < cols; c += kThreads) {
      const float d = load_one<DT>(v, at + c) - mean;
      q += d * d;
    }
    const float rstd = static_cast<float>(1.0 / sqrt(static_cast<double>(cta_sum(q, 0.f).x / n) + a.eps));
    for (uint32_t c = threadIdx.x; c < cols; c += kThreads) {
      const float b = a.bias[r] != nullptr ? load_one<WT>(a.bias[r], c) : 0.f;
      save_one<DT>(a.out[r], at + c, (load_one<DT>(v, at + c) - mean) * rstd * load_one<WT>(a.weight[r], c) + b);
    }
    if (threadIdx.x == 0 && a.mean[r] != nullptr) {
      a.mean[r][row] = mean;
      a.rstd[r][row] = rstd;
    }
  }
}

template <int DT, int WT>
__global__ void __launch_bounds__(kThreads) norm_grad_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ float acc[];  // cols sums for the weight, then for the bias
  pdl_enter();
  const RowPart part = row_part(a.parts, a.p, blockIdx.x);
  const int r = part.r;
  const uint32_t cols = a.cols;
  const float n = static_cast<float>(cols);
  for (uint32_t c = threadIdx.x; c < 2 * cols; c += kThreads) acc[c] = 0.f;
  __syncthreads();
  for (uint32_t row = part.lo; row < part.hi; ++row) {
    const uint64_t at = static_cast<uint64_t>(row) * cols;
    const float mean = a.mean[r][row], rstd = a.rstd[r][row];
    float sg = 0.f, sgz = 0.f;
    for (uint32_t c = threadIdx.x; c < cols; c += kThreads) {
      const float d = load_one<DT>(a.dy[r], at + c), z = (load_one<DT>(a.x[r], at + c) - mean) * rstd;
      const float g = d * load_one<WT>(a.weight[r], c);
      sg += g;
      sgz += g * z;
      acc[c] += d * z;
      acc[cols + c] += d;
    }
    const float2 t = cta_sum(sg, sgz);
    for (uint32_t c = threadIdx.x; c < cols; c += kThreads) {
      const float z = (load_one<DT>(a.x[r], at + c) - mean) * rstd;
      const float g = load_one<DT>(a.dy[r], at + c) * load_one<WT>(a.weight[r], c);
      const float more = a.extra[r] != nullptr ? load_one<DT>(a.extra[r], at + c) : 0.f;
      save_one<DT>(a.out[r], at + c, (g - t.x / n - z * (t.y / n)) * rstd + more);
    }
  }
  if (a.partial == nullptr) return;
  float* out = a.partial + static_cast<uint64_t>(blockIdx.x) * 2 * cols;
  __syncthreads();
  for (uint32_t c = threadIdx.x; c < 2 * cols; c += kThreads) out[c] = acc[c];
}

// A rank's parts added up (grid y = rank).
template <int DT>
__global__ void __launch_bounds__(kThreads) norm_join_kernel(const __grid_constant__ NormJoinArgs a) {
  pdl_enter();
  const int r = blockIdx.y;
  const uint32_t c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= a.cols) return;
  float w = 0.f, b = 0.f;
  for (uint32_t i = a.first[r]; i < a.first[r + 1]; ++i) {
    const float* part = a.partial + static_cast<uint64_t>(i) * 2 * a.cols;
    w += part[c];
    b += part[a.cols + c];
  }
  if (a.weight) save_one<DT>(a.dweight[r], c, w);
  if (a.bias) save_one<DT>(a.dbias[r], c, b);
}

template <typename F>
cudaError_t by_types(int dt, int wt, F f) {
  const auto with = [&](auto d) {
    return wt == kF32 ? f(d, std::integral_constant<int, kF32>{}) : f(d, std::integral_constant<int, kBF16>{});
  };
  return dt == kF32 ? with(std::integral_constant<int, kF32>{}) : with(std::integral_constant<int, kBF16>{});
}

}  // namespace

cudaError_t launch_norm(int dt, int weight_dt, bool, const NormArgs& a, cudaStream_t s) {
  return by_types(dt, weight_dt, [&](auto d, auto w) {
    const cudaError_t err = launch_kernel(norm_kernel<decltype(d)::value, decltype(w)::value>, dim3(a.parts.first[a.p]), dim3(kThreads), s, a);
    if (err == cudaSuccess) note_launch();
    return err;
  });
}

cudaError_t launch_norm_grad(int dt, int weight_dt, bool, bool, const NormArgs& a, cudaStream_t s) {
  return by_types(dt, weight_dt, [&](auto d, auto w) {
    auto* kernel = norm_grad_kernel<decltype(d)::value, decltype(w)::value>;
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kNormMaxCols * 8));
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.parts.first[a.p]);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = a.cols * 8;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = CCL_PDL ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, kernel, a);
    if (err == cudaSuccess) note_launch();
    return err;
  });
}

cudaError_t launch_norm_join(int dw_dt, const NormJoinArgs& a, cudaStream_t s) {
  const dim3 grid((a.cols + kThreads - 1) / kThreads, static_cast<unsigned>(a.p));
  const cudaError_t err = dw_dt == kF32 ? launch_kernel(norm_join_kernel<kF32>, grid, dim3(kThreads), s, a)
                                        : launch_kernel(norm_join_kernel<kBF16>, grid, dim3(kThreads), s, a);
  if (err == cudaSuccess) note_launch();
  return err;
}

}  // namespace ccl
