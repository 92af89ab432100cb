// adamw.cu -- one AdamW step over many tensors, states in 32 or 8 bits.
//
// Per element (include/ccl.h has the formula): read the parameter, its
// gradient and two moments, write the parameter and the moments, every
// operation rounded to fp32 by itself so that the result does not depend on
// how the compiler contracts it.  Bound by HBM: 26 bytes per element with
// fp32 parameters and states and bf16 gradients, 14.125 with 8-bit states.
//
// An 8-bit state is e4m3 codes with one fp32 scale per 128 elements.  A warp
// holds such a block with four elements per lane, so its amax is one
// warp-wide integer maximum of the magnitudes' bits.
#include <cuda_fp8.h>

#include "device_common.cuh"

namespace ccl {
namespace {

constexpr int kPer = 4;                                   // elements per lane
constexpr int kBlocksPerWarp = kAdamwChunk / kAdamwBlock / (kThreads / 32);  // 4
constexpr uint32_t kDitherElem = 1779033703u;

// Four consecutive elements of type DT at element i, fp32, through one vector
// where the tensor's addresses allow it (`vec`); elements from n on are 0.
template <int DT>
__device__ __forceinline__ void load4(const void* base, uint64_t i, uint64_t n, bool vec, float* x) {
  if (vec && i + kPer <= n) {
    if constexpr (DT == kF32) {
      const uint4 v = ld_once16(static_cast<const char*>(base) + i * 4);
      x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
    } else {
      const uint2 v = __ldcs(reinterpret_cast<const uint2*>(static_cast<const char*>(base) + i * 2));
      x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xFFFF0000u);
      x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
    return;
  }
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    x[q] = 0.0f;
    if (i + q < n) {
      if constexpr (DT == kF32) x[q] = __uint_as_float(ld_once4(static_cast<const char*>(base) + (i + q) * 4));
      else x[q] = __uint_as_float(ld_once2(static_cast<const char*>(base) + (i + q) * 2) << 16);
    }
  }
}
template <int DT>
__device__ __forceinline__ void store4(void* base, uint64_t i, uint64_t n, bool vec, const float* x) {
  uint32_t w[kPer];
  if (vec && i + kPer <= n) {
    pack_out<DT, kPer>(x, w);
    if constexpr (DT == kF32) st_stream16(static_cast<char*>(base) + i * 4, make_uint4(w[0], w[1], w[2], w[3]));
    else __stcs(reinterpret_cast<uint2*>(static_cast<char*>(base) + i * 2), make_uint2(w[0], w[1]));
    return;
  }
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    if (i + q >= n) continue;
    pack_out<DT, 1>(x + q, w);
    store_one<DT>(base, i + q, w, 0);
  }
}

__device__ __forceinline__ uint32_t load_codes(const void* base, uint64_t i, uint64_t n, bool vec) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + i;
  if (vec && i + kPer <= n) return ld_once4(p);
  uint32_t w = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q)
    if (i + q < n) w |= static_cast<uint32_t>(p[q]) << (8 * q);
  return w;
}
__device__ __forceinline__ void store_codes(void* base, uint64_t i, uint64_t n, bool vec, uint32_t w) {
  uint8_t* p = static_cast<uint8_t*>(base) + i;
  if (vec && i + kPer <= n) {
    st_stream4(p, w);
    return;
  }
#pragma unroll
  for (int q = 0; q < kPer; ++q)
    if (i + q < n) p[q] = static_cast<uint8_t>(w >> (8 * q));
}

// Four e4m3 codes to fp32 (exact).
__device__ __forceinline__ void decode4(uint32_t w, float* x) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw v = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * h)), __NV_E4M3);
    const float2 f = __half22float2(__half2(v));
    x[2 * h] = f.x, x[2 * h + 1] = f.y;
  }
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// The block's amax over finite values (bits of non-negative floats compare as
// integers), its scale and the factor that codes are made with.
__device__ __forceinline__ void block_scale(const float* x, float* up, float* scale) {
  uint32_t top = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) top = max(top, finite(x[q]) ? __float_as_uint(fabsf(x[q])) : 0u);
  const float amax = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, top));
  const bool some = amax > 7.888609052210118e-31f;  // 2^-100
  *up = some ? __fmul_rn(__frcp_rn(amax), 448.0f) : 0.0f;
  *scale = some ? __fmul_rn(amax, 1.0f / 448.0f) : 1.0f;
}

template <int PDT, int GDT, int BITS, bool COPY, typename Args>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Args a) {
  pdl_enter();
  // the tensor of this chunk: the last whose first chunk is not past it
  int lo = 0, hi = a.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.chunk0[mid] <= blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const AdamwTensor t = a.t[lo];
  const uint64_t c0 = static_cast<uint64_t>(blockIdx.x - a.chunk0[lo]) * kAdamwChunk;
  const uint64_t n = t.n;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool pv = (reinterpret_cast<uintptr_t>(t.param) & (PDT == kF32 ? 15 : 7)) == 0;
  const bool gv = (reinterpret_cast<uintptr_t>(t.grad) & (GDT == kF32 ? 15 : 7)) == 0;
  const bool sv = ((reinterpret_cast<uintptr_t>(t.m) | reinterpret_cast<uintptr_t>(t.v)) & (BITS == 32 ? 15 : 3)) == 0;
  const bool cv = COPY && (reinterpret_cast<uintptr_t>(t.copy) & 7) == 0;
  const float grad_scale = a.grad_scale != nullptr ? *a.grad_scale : 1.0f;
#pragma unroll
  for (int b = 0; b < kBlocksPerWarp; ++b) {
    const uint64_t i0 = c0 + static_cast<uint64_t>(b * (kThreads / 32) + warp) * kAdamwBlock;
    if (i0 >= n) continue;  // the whole warp
    const uint64_t i = i0 + lane * kPer, block = i0 / kAdamwBlock;
    float p[kPer], g[kPer], m[kPer], v[kPer];
    load4<PDT>(t.param, i, n, pv, p);
    load4<GDT>(t.grad, i, n, gv, g);
    if constexpr (BITS == 32) {
      load4<kF32>(t.m, i, n, sv, m);
      load4<kF32>(t.v, i, n, sv, v);
    } else {
      const uint32_t mc = load_codes(t.m, i, n, sv), vc = load_codes(t.v, i, n, sv);
      const float ms = t.m_scale[block], vs = t.v_scale[block];
      decode4(mc, m);
      decode4(vc, v);
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        m[q] = __fmul_rn(m[q], ms);
        v[q] = __fmul_rn(v[q], vs);
        v[q] = __fmul_rn(v[q], v[q]);
      }
    }
    float root[kPer];
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const float gq = a.grad_scale != nullptr ? __fmul_rn(g[q], grad_scale) : g[q];
      m[q] = __fadd_rn(__fmul_rn(m[q], a.beta1), __fmul_rn(gq, a.one_minus_beta1));
      v[q] = __fadd_rn(__fmul_rn(v[q], a.beta2), __fmul_rn(__fmul_rn(gq, gq), a.one_minus_beta2));
      root[q] = __fsqrt_rn(v[q]);
      const float den = __fadd_rn(__fmul_rn(root[q], a.root_scale), a.eps);
      p[q] = __fsub_rn(__fmul_rn(p[q], a.decay), __fmul_rn(__fdiv_rn(m[q], den), a.step_size));
    }
    store4<PDT>(t.param, i, n, pv, p);
    if constexpr (COPY)
      if (t.copy != nullptr) store4<kBF16>(t.copy, i, n, cv, p);
    if constexpr (BITS == 32) {
      store4<kF32>(t.m, i, n, sv, m);
      store4<kF32>(t.v, i, n, sv, v);
    } else {
      float mu, ms, vu, vs;
      block_scale(m, &mu, &ms);
      block_scale(root, &vu, &vs);
      uint32_t mc = 0, vc = 0;
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        uint32_t code = __nv_cvt_float_to_fp8(__fmul_rn(m[q], mu), __NV_SATFINITE, __NV_E4M3);
        if (!finite(m[q])) code = 0x7F;
        mc |= code << (8 * q);
        // an e4m3 number times 2^-120 has its code in the top bits of its
        // fp32 form, subnormals included; the threshold below the last code
        // bit makes the carry that rounds up
        const uint32_t threshold = (static_cast<uint32_t>(i + q) * kDitherElem + a.dither) >> 12;
        const float x = __fmul_rn(__fmul_rn(root[q], vu), 7.52316384526264e-37f);  // 2^-120
        code = min((__float_as_uint(x) + threshold) >> 20, 0x7Eu);
        code = vu > 0.0f ? (v[q] > 0.0f ? max(code, 1u) : code) : 0u;
        if (!finite(root[q])) code = 0x7F;
        vc |= code << (8 * q);
      }
      store_codes(t.m, i, n, sv, mc);
      store_codes(t.v, i, n, sv, vc);
      if (lane == 0) {
        t.m_scale[block] = ms;
        t.v_scale[block] = vs;
      }
    }
  }
}

template <int PDT, int GDT, int BITS, bool COPY, typename Args>
cudaError_t launch_one(const Args& a, cudaStream_t s) {
  return launch_kernel(adamw_kernel<PDT, GDT, BITS, COPY, Args>, dim3(a.chunk0[a.count]), dim3(kThreads), s, a);
}

template <int PDT, int GDT, typename Args>
cudaError_t launch_types(int bits, bool copy, const Args& a, cudaStream_t s) {
  if constexpr (PDT == kF32) {
    if (copy) return bits == 8 ? launch_one<PDT, GDT, 8, true>(a, s) : launch_one<PDT, GDT, 32, true>(a, s);
  }
  return bits == 8 ? launch_one<PDT, GDT, 8, false>(a, s) : launch_one<PDT, GDT, 32, false>(a, s);
}

template <typename Args>
cudaError_t launch_any(int pdt, int gdt, int bits, bool copy, const Args& a, cudaStream_t s) {
  if (a.chunk0[a.count] == 0) return cudaSuccess;
  cudaError_t err = pdt == kF32 ? (gdt == kF32 ? launch_types<kF32, kF32>(bits, copy, a, s) : launch_types<kF32, kBF16>(bits, copy, a, s))
                                : (gdt == kF32 ? launch_types<kBF16, kF32>(bits, copy, a, s) : launch_types<kBF16, kBF16>(bits, copy, a, s));
  if (err == cudaSuccess) note_launch();
  return err;
}

}  // namespace

cudaError_t launch_adamw(int param_dt, int grad_dt, int bits, bool copy, const AdamwSmall& a, cudaStream_t s) {
  return launch_any(param_dt, grad_dt, bits, copy, a, s);
}
cudaError_t launch_adamw(int param_dt, int grad_dt, int bits, bool copy, const AdamwLarge& a, cudaStream_t s) {
  return launch_any(param_dt, grad_dt, bits, copy, a, s);
}

}  // namespace ccl
