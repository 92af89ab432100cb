// moe_product.cu -- the experts' products: each expert's rows times its
// weights, and the gradients for the rows and for the weights.
#include "device_common.cuh"

namespace ccl {
namespace {

constexpr int kTile = 64, kStep = 16;

// 64 x 64 tile of one expert's product, 4 x 4 outputs per thread, operands
// staged element by element in shared memory as fp32.  grid.x walks the
// output columns, grid.y the row tiles of all experts (each expert starts
// tiles of its own; the weights' gradient has the same tiles for each),
// grid.z the ranks.
template <int KIND, int OUT>
__global__ void __launch_bounds__(kThreads) product_simple_kernel(const __grid_constant__ ProductArgs a) {
  __shared__ float as[kStep][kTile + 1], bs[kStep][kTile + 1];
  pdl_enter();
  const int r = blockIdx.z, E = a.num_experts;
  const int32_t* off = a.offsets[r];
  const int64_t rows = a.rows[r], N = a.n, K = a.contract;
  int e = 0;
  int64_t tile = blockIdx.y, lo = 0, hi = 0;
  const int64_t wt = (N + kTile - 1) / kTile;
  for (; e < E; ++e) {  // the expert of this tile
    lo = min(max(static_cast<int64_t>(off[e]), int64_t{0}), rows);
    hi = min(max(static_cast<int64_t>(off[e + 1]), lo), rows);
    const int64_t tiles = KIND == kProductGradWeight ? wt : (hi - lo + kTile - 1) / kTile;
    if (tile < tiles) break;
    tile -= tiles;
  }
  if (e == E) return;
  const int64_t m0 = tile * kTile, n0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const int64_t M = KIND == kProductGradWeight ? N : hi - lo;
  const int64_t cols = KIND == kProductForward ? N : K;
  const int64_t depth = KIND == kProductForward ? K : KIND == kProductGradInput ? N : hi - lo;
  const __nv_bfloat16* A = static_cast<const __nv_bfloat16*>(a.a[r]);
  const __nv_bfloat16* B = static_cast<const __nv_bfloat16*>(a.b[r]);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < depth; k0 += kStep) {
    for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
      // consecutive threads along the operand's contiguous axis
      const int ak = KIND == kProductGradWeight ? i / kTile : i % kStep, am = KIND == kProductGradWeight ? i % kTile : i / kStep;
      float v = 0.0f;
      if (m0 + am < M && k0 + ak < depth)
        v = __bfloat162float(KIND == kProductGradWeight ? A[(lo + k0 + ak) * N + m0 + am] : A[(lo + m0 + am) * depth + k0 + ak]);
      as[ak][am] = v;
      const int bk = KIND == kProductForward ? i % kStep : i / kTile, bn = KIND == kProductForward ? i / kStep : i % kTile;
      v = 0.0f;
      if (n0 + bn < cols && k0 + bk < depth)
        v = __bfloat162float(KIND == kProductForward     ? B[(e * N + n0 + bn) * K + k0 + bk]
                             : KIND == kProductGradInput ? B[(e * N + k0 + bk) * K + n0 + bn]
                                                         : B[(lo + k0 + bk) * K + n0 + bn]);
      bs[bk][bn] = v;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < kStep; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(as[kk][ty * 4 + i], bs[kk][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i, n = n0 + tx + 16 * j;
      if (m >= M || n >= cols) continue;
      const int64_t at = ((KIND == kProductGradWeight ? e * N : lo) + m) * cols + n;
      if constexpr (OUT == kF32) static_cast<float*>(a.out[r])[at] = acc[i][j];
      else static_cast<__nv_bfloat16*>(a.out[r])[at] = __float2bfloat16_rn(acc[i][j]);
    }
  }
}

}  // namespace

cudaError_t launch_moe_product(int kind, int out_dt, const ProductArgs& a, cudaStream_t s) {
  uint64_t most = 0;
  for (int r = 0; r < a.p; ++r) most = a.rows[r] > most ? a.rows[r] : most;
  const uint64_t cols = kind == kProductForward ? a.n : a.contract;
  const uint64_t gy = kind == kProductGradWeight ? a.num_experts * ((a.n + kTile - 1) / kTile) : (most + kTile - 1) / kTile + a.num_experts;
  const dim3 grid(static_cast<unsigned>((cols + kTile - 1) / kTile), static_cast<unsigned>(gy), static_cast<unsigned>(a.p));
  cudaError_t err = kind == kProductForward     ? launch_kernel(product_simple_kernel<kProductForward, kBF16>, grid, dim3(kThreads), s, a)
                    : kind == kProductGradInput ? launch_kernel(product_simple_kernel<kProductGradInput, kBF16>, grid, dim3(kThreads), s, a)
                    : out_dt == kF32            ? launch_kernel(product_simple_kernel<kProductGradWeight, kF32>, grid, dim3(kThreads), s, a)
                                                : launch_kernel(product_simple_kernel<kProductGradWeight, kBF16>, grid, dim3(kThreads), s, a);
  if (err == cudaSuccess) note_launch();
  return err;
}

}  // namespace ccl
