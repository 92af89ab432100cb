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

constexpr int kPer = 4;  // elements per lane: a warp holds a block of 128
constexpr int kBlocksPerWarp = kAdamwChunk / kAdamwBlock / (kThreads / 32);
constexpr uint32_t kDitherElem = 1779033703u;
constexpr uint32_t kInf = 0x7F800000u;

// Four consecutive elements of type DT as they lie in memory, from element i
// of n: through one vector where the tensor's address allows it (`vec`),
// zeros from n on.
template <int DT>
struct Raw4 {
  uint32_t w[DT == kF32 ? 4 : 2];
};
template <int DT>
__device__ __forceinline__ void load4(const void* base, uint64_t i, uint64_t n, bool vec, Raw4<DT>& r) {
  const char* p = static_cast<const char*>(base) + i * Elem<DT>::kBytes;
  if (vec && i + kPer <= n) {
    if constexpr (DT == kF32) {
      const uint4 v = ld_once16(p);
      r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
    } else {
      const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
      r.w[0] = v.x, r.w[1] = v.y;
    }
    return;
  }
  if constexpr (DT == kF32) {
#pragma unroll
    for (int q = 0; q < kPer; ++q) r.w[q] = i + q < n ? ld_once4(p + 4 * q) : 0u;
  } else {
#pragma unroll
    for (int q = 0; q < kPer; q += 2)
      r.w[q / 2] = (i + q < n ? ld_once2(p + 2 * q) : 0u) | (i + q + 1 < n ? ld_once2(p + 2 * q + 2) << 16 : 0u);
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

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// The block's amax over finite values (bits of magnitudes compare as
// integers), its scale and the factor that codes are made with.  Returns
// whether every value is finite, which is all but always so.
__device__ __forceinline__ bool block_scale(const float* x, float* up, float* scale) {
  uint32_t top = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) top = max(top, magnitude(x[q]));
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  const bool fine = top < kInf;
  if (!fine) {
    top = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) top = max(top, magnitude(x[q]) < kInf ? magnitude(x[q]) : 0u);
    top = __reduce_max_sync(0xFFFFFFFFu, top);
  }
  const float amax = __uint_as_float(top);
  const bool some = amax > 7.888609052210118e-31f;  // 2^-100
  *up = some ? __fmul_rn(__frcp_rn(amax), 448.0f) : 0.0f;
  *scale = some ? __fmul_rn(amax, 1.0f / 448.0f) : 1.0f;
  return fine;
}

// `codes` with 0x7F (NaN) where a value is not finite.
__device__ __forceinline__ uint32_t mark_not_finite(uint32_t codes, const float* x) {
#pragma unroll
  for (int q = 0; q < kPer; ++q)
    if (magnitude(x[q]) >= kInf) codes |= 0x7Fu << (8 * q), codes &= ~(0x80u << (8 * q));
  return codes;
}

// A block's inputs, loaded together before any is used: with 8-bit states a
// block is 14 bytes a lane-element less than with fp32 ones, so more blocks
// have to be in flight for the same bandwidth.
template <int PDT, int GDT, int BITS>
struct Inputs {
  Raw4<PDT> p;
  Raw4<GDT> g;
  Raw4<kF32> m, v;       // BITS == 32
  uint32_t mc, vc;       // BITS == 8
  float ms, vs;
};

template <int PDT, int GDT, int BITS, bool COPY, typename Args>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Args a) {
  constexpr int U = BITS == 8 ? 4 : 2;  // blocks in flight per warp
  static_assert(kBlocksPerWarp % U == 0, "whole batches");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // the tensor of this chunk: the last whose first chunk is not past it
  int at = -1;
  for (int i = 0; i < a.count; i += 32)
    at += __popc(__ballot_sync(0xFFFFFFFFu, i + lane < a.count && a.chunk0[min(i + lane, a.count)] <= blockIdx.x));
  const AdamwTensor& t = a.t[at];
  const uint64_t c0 = static_cast<uint64_t>(blockIdx.x - a.chunk0[at]) * kAdamwChunk;
  const uint64_t n = t.n;
  const bool pv = (reinterpret_cast<uintptr_t>(t.param) & (PDT == kF32 ? 15 : 7)) == 0;
  const bool gv = (reinterpret_cast<uintptr_t>(t.grad) & (GDT == kF32 ? 15 : 7)) == 0;
  const bool sv = ((reinterpret_cast<uintptr_t>(t.m) | reinterpret_cast<uintptr_t>(t.v)) & (BITS == 32 ? 15 : 3)) == 0;
  const bool cv = COPY && (reinterpret_cast<uintptr_t>(t.copy) & 7) == 0;
  pdl_enter();
  const float grad_scale = a.grad_scale != nullptr ? *a.grad_scale : 1.0f;
#pragma unroll
  for (int b0 = 0; b0 < kBlocksPerWarp; b0 += U) {
    Inputs<PDT, GDT, BITS> in[U];
#pragma unroll
    for (int b = 0; b < U; ++b) {
      const uint64_t i0 = c0 + static_cast<uint64_t>((b0 + b) * (kThreads / 32) + warp) * kAdamwBlock;
      if (i0 >= n) continue;  // the whole warp
      const uint64_t i = i0 + lane * kPer, block = i0 / kAdamwBlock;
      load4<PDT>(t.param, i, n, pv, in[b].p);
      load4<GDT>(t.grad, i, n, gv, in[b].g);
      if constexpr (BITS == 32) {
        load4<kF32>(t.m, i, n, sv, in[b].m);
        load4<kF32>(t.v, i, n, sv, in[b].v);
      } else {
        in[b].mc = load_codes(t.m, i, n, sv);
        in[b].vc = load_codes(t.v, i, n, sv);
        in[b].ms = t.m_scale[block];
        in[b].vs = t.v_scale[block];
      }
    }
#pragma unroll
    for (int b = 0; b < U; ++b) {
      const uint64_t i0 = c0 + static_cast<uint64_t>((b0 + b) * (kThreads / 32) + warp) * kAdamwBlock;
      if (i0 >= n) continue;
      const uint64_t i = i0 + lane * kPer, block = i0 / kAdamwBlock;
      float p[kPer], m[kPer], v[kPer], root[kPer];
      if constexpr (BITS == 32) {
#pragma unroll
        for (int q = 0; q < kPer; ++q) m[q] = widen<kF32>(in[b].m.w, q), v[q] = widen<kF32>(in[b].v.w, q);
      } else {
        decode4(in[b].mc, m);
        decode4(in[b].vc, v);
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
          m[q] = __fmul_rn(m[q], in[b].ms);
          v[q] = __fmul_rn(v[q], in[b].vs);
          v[q] = __fmul_rn(v[q], v[q]);
        }
      }
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        float g = widen<GDT>(in[b].g.w, q);
        if (a.grad_scale != nullptr) g = __fmul_rn(g, grad_scale);
        m[q] = __fadd_rn(__fmul_rn(m[q], a.beta1), __fmul_rn(g, a.one_minus_beta1));
        v[q] = __fadd_rn(__fmul_rn(v[q], a.beta2), __fmul_rn(__fmul_rn(g, g), a.one_minus_beta2));
        root[q] = __fsqrt_rn(v[q]);
        const float den = __fadd_rn(__fmul_rn(root[q], a.root_scale), a.eps);
        p[q] = __fsub_rn(__fmul_rn(widen<PDT>(in[b].p.w, q), a.decay), __fmul_rn(__fdiv_rn(m[q], den), a.step_size));
      }
      store4<PDT>(t.param, i, n, pv, p);
      if constexpr (COPY)
        if (t.copy != nullptr) store4<kBF16>(t.copy, i, n, cv, p);
      if constexpr (BITS == 32) {
        store4<kF32>(t.m, i, n, sv, m);
        store4<kF32>(t.v, i, n, sv, v);
      } else {
        float mu, ms, vu, vs;
        const bool fine = block_scale(m, &mu, &ms) & block_scale(root, &vu, &vs);
        uint32_t mc = 0, vc = 0;
#pragma unroll
        for (int q = 0; q < kPer; q += 2)
          mc |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(m[q], mu), __fmul_rn(m[q + 1], mu)),
                                                               __NV_SATFINITE, __NV_E4M3)) << (8 * q);
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
          // an e4m3 number times 2^-120 has its code in the top bits of its
          // fp32 form, subnormals included; the threshold below the last code
          // bit makes the carry that rounds up.  A code of 0 is a 1 where v is
          // not 0 (with vu = 0 the block holds nothing worth a code).
          const uint32_t threshold = (static_cast<uint32_t>(i + q) * kDitherElem + a.dither) >> 12;
          const float x = __fmul_rn(__fmul_rn(root[q], vu), 7.52316384526264e-37f);  // 2^-120
          const uint32_t least = v[q] > 0.0f && vu > 0.0f ? 1u : 0u;
          const uint32_t code = vu > 0.0f ? (__float_as_uint(x) + threshold) >> 20 : 0u;
          vc |= max(min(code, 0x7Eu), least) << (8 * q);
        }
        if (!fine) mc = mark_not_finite(mc, m), vc = mark_not_finite(vc, root);
        store_codes(t.m, i, n, sv, mc);
        store_codes(t.v, i, n, sv, vc);
        if (lane == 0) {
          t.m_scale[block] = ms;
          t.v_scale[block] = vs;
        }
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
