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

// ------------------------------------------------------- elements of a lane
// VEC: lane l holds elements 4 l .. 4 l + 3 of the block, by one vector access
// (every array of the tensor on the vector's grid).  Otherwise elements l,
// l + 32, l + 64, l + 96, so that each of the four accesses of a warp is one
// contiguous run wherever the array starts; with four neighbours per lane the
// scalar accesses of an array off the grid asked L2 for every sector four
// times (157 M elements with 8-bit states 869 us against 696 on the grid).
template <bool VEC>
__device__ __forceinline__ int element(int lane, int q) {
  return VEC ? lane * kPer + q : lane + 32 * q;
}

template <int DT>
struct Raw4 {
  uint32_t w[kPer];  // VEC: as loaded; else element q in the low bits of w[q]
};
// Elements of the block at `base` + i0, of which `count` (up to 128) exist; zeros behind them.
template <int DT, bool VEC>
__device__ __forceinline__ void load4(const void* base, uint64_t i0, int lane, int count, Raw4<DT>& r) {
  const char* p = static_cast<const char*>(base) + i0 * Elem<DT>::kBytes;
  if constexpr (VEC) {
    if (lane * kPer + kPer <= count) {
      if constexpr (DT == kF32) {
        const uint4 v = ld_once16(p + lane * 16);
        r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
      } else {
        const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p + lane * 8));
        r.w[0] = v.x, r.w[1] = v.y;
      }
      return;
    }
  }
  uint32_t e[kPer];
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int i = element<VEC>(lane, q);
    e[q] = i >= count ? 0u : DT == kF32 ? ld_once4(p + i * 4) : ld_once2(p + i * 2);
  }
  if constexpr (VEC && DT == kBF16) {
    r.w[0] = e[0] | e[1] << 16, r.w[1] = e[2] | e[3] << 16;
  } else {
#pragma unroll
    for (int q = 0; q < kPer; ++q) r.w[q] = e[q];
  }
}
template <int DT, bool VEC>
__device__ __forceinline__ float value(const Raw4<DT>& r, int q) {
  if constexpr (VEC || DT == kF32) return widen<DT>(r.w, q);
  else return __uint_as_float(r.w[q] << 16);
}
template <int DT, bool VEC>
__device__ __forceinline__ void store4(void* base, uint64_t i0, int lane, int count, const float* x) {
  char* p = static_cast<char*>(base) + i0 * Elem<DT>::kBytes;
  uint32_t w[kPer];
  if constexpr (VEC) {
    if (lane * kPer + kPer <= count) {
      pack_out<DT, kPer>(x, w);
      if constexpr (DT == kF32) st_stream16(p + lane * 16, make_uint4(w[0], w[1], w[2], w[3]));
      else __stcs(reinterpret_cast<uint2*>(p + lane * 8), make_uint2(w[0], w[1]));
      return;
    }
  }
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int i = element<VEC>(lane, q);
    if (i >= count) continue;
    pack_out<DT, 1>(x + q, w);
    store_one<DT>(p, i, w, 0);
  }
}
template <bool VEC>
__device__ __forceinline__ uint32_t load_codes(const void* base, uint64_t i0, int lane, int count) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + i0;
  if (VEC && lane * kPer + kPer <= count) return ld_once4(p + lane * kPer);
  uint32_t w = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int i = element<VEC>(lane, q);
    if (i < count) w |= static_cast<uint32_t>(__ldcs(p + i)) << (8 * q);
  }
  return w;
}
template <bool VEC>
__device__ __forceinline__ void store_codes(void* base, uint64_t i0, int lane, int count, uint32_t w) {
  uint8_t* p = static_cast<uint8_t*>(base) + i0;
  if (VEC && lane * kPer + kPer <= count) {
    st_stream4(p + lane * kPer, w);
    return;
  }
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int i = element<VEC>(lane, q);
    if (i < count) __stcs(p + i, static_cast<uint8_t>(w >> (8 * q)));
  }
}

// ------------------------------------------------------- pairs of fp32 numbers
// One instruction, two operations, each rounded to nearest as the single ones
// are.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 pair(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 both(float a) { return pair(a, a); }
__device__ __forceinline__ float2 parts(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// a + b, where a is a product that was rounded by itself.  `one` is 1, but the
// assembler must not know: it joined paired products with paired sums behind
// them, for all that both name their rounding, and the product's was lost.
__device__ __forceinline__ F2 add2(F2 a, F2 b, F2 one) { return fma2(a, one, b); }
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Square root and quotient rounded to nearest, from an approximate reciprocal
// (square root) and fused multiply-adds: Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor" (1990), and Cornea,
// Harrison and Tang, "Scientific Computing on Itanium-based Systems" (2002).
// One refinement of the approximation, a residual that the fused operation
// makes exact, one correction.  The residuals stay exact while the operands
// keep away from the ends of the exponent range (nonzero operands in 2^-95 .. 2^40, which is checked); two
// numbers take 8 and 6 paired instructions.
__device__ __forceinline__ F2 sqrt2(F2 x) {
  const float2 s = parts(x);
  const F2 y = pair(s.x > 0.0f ? rsqrt_approx(s.x) : 0.0f, s.y > 0.0f ? rsqrt_approx(s.y) : 0.0f);
  F2 g = mul2(x, y), nh = mul2(y, both(-0.5f));  // sqrt(x) and -1 / (2 sqrt(x)), nearly
  const F2 r = fma2(nh, g, both(0.5f));
  g = fma2(g, r, g);
  nh = fma2(nh, r, nh);
  const F2 d = fma2(g, g, mul2(x, both(-1.0f)));  // g^2 - x, exact
  return fma2(nh, d, g);
}
__device__ __forceinline__ F2 div2(F2 a, F2 b) {
  const float2 s = parts(b);
  F2 y = pair(rcp_approx(s.x), rcp_approx(s.y));
  const F2 nb = mul2(b, both(-1.0f));
  y = fma2(fma2(nb, y, both(1.0f)), y, y);
  const F2 q = mul2(a, y);
  return fma2(fma2(nb, q, a), y, q);  // q + (a - b q) / b, the residual exact
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
constexpr uint32_t kLeast = (127u - 95u) << 23, kMost = (127u + 40u) << 23;  // 2^-95 and 2^40

// ------------------------------------------------------------- 8-bit states
// Four e4m3 codes to fp32 (exact).
__device__ __forceinline__ void decode4(uint32_t w, F2* x) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw v = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * h)), __NV_E4M3);
    const float2 f = __half22float2(__half2(v));
    x[h] = pair(f.x, f.y);
  }
}

// From the bits of a block's largest finite magnitude: the factor that codes
// are made with, and the scale.
__device__ __forceinline__ void block_scale(uint32_t top, float* up, float* scale) {
  const float amax = __uint_as_float(top);
  const bool some = amax > 7.888609052210118e-31f;  // 2^-100
  *up = some ? __fmul_rn(__frcp_rn(amax), 448.0f) : 0.0f;
  *scale = some ? __fmul_rn(amax, 1.0f / 448.0f) : 1.0f;
}

// The block's largest finite magnitude, for blocks that hold other values too.
__device__ __forceinline__ uint32_t finite_top(const float* x) {
  uint32_t top = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) top = max(top, magnitude(x[q]) < kInf ? magnitude(x[q]) : 0u);
  return __reduce_max_sync(0xFFFFFFFFu, top);
}

// `codes` with 0x7F (NaN) where a value is not finite.
__device__ __forceinline__ uint32_t mark_not_finite(uint32_t codes, const float* x) {
#pragma unroll
  for (int q = 0; q < kPer; ++q)
    if (magnitude(x[q]) >= kInf) codes = (codes & ~(0xFFu << (8 * q))) | 0x7Fu << (8 * q);
  return codes;
}

template <int PDT, int GDT, int BITS>
struct Inputs {
  Raw4<PDT> p;
  Raw4<GDT> g;
  Raw4<kF32> m, v;  // BITS == 32
  uint32_t mc, vc;  // BITS == 8
  float ms, vs;
};

// A chunk of one tensor: warp w takes blocks w, w + 8, ..., U of them loaded
// together before any is used, so that enough bytes are on their way.
template <int PDT, int GDT, int BITS, bool COPY, bool VEC, typename Args>
__device__ __forceinline__ void adamw_chunk(const Args& a, const AdamwTensor& t, uint64_t c0, float grad_scale) {
  constexpr int U = 2;
  static_assert(kBlocksPerWarp % U == 0, "whole batches");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t n = t.n;
  const F2 one = both(a.one);
#pragma unroll 1
  for (int b0 = 0; b0 < kBlocksPerWarp; b0 += U) {
    const uint64_t first = c0 + static_cast<uint64_t>(b0 * (kThreads / 32) + warp) * kAdamwBlock;
    if (first >= n) return;  // the whole warp
    Inputs<PDT, GDT, BITS> in[U];
#pragma unroll
    for (int b = 0; b < U; ++b) {
      const uint64_t i0 = first + b * (kThreads / 32) * kAdamwBlock;
      if (i0 >= n) continue;
      const int count = static_cast<int>(min(n - i0, static_cast<uint64_t>(kAdamwBlock)));
      load4<PDT, VEC>(t.param, i0, lane, count, in[b].p);
      load4<GDT, VEC>(t.grad, i0, lane, count, in[b].g);
      if constexpr (BITS == 32) {
        load4<kF32, VEC>(t.m, i0, lane, count, in[b].m);
        load4<kF32, VEC>(t.v, i0, lane, count, in[b].v);
      } else {
        in[b].mc = load_codes<VEC>(t.m, i0, lane, count);
        in[b].vc = load_codes<VEC>(t.v, i0, lane, count);
        in[b].ms = t.m_scale[i0 / kAdamwBlock];
        in[b].vs = t.v_scale[i0 / kAdamwBlock];
      }
    }
#pragma unroll
    for (int b = 0; b < U; ++b) {
      const uint64_t i0 = first + b * (kThreads / 32) * kAdamwBlock;
      if (i0 >= n) continue;
      const int count = static_cast<int>(min(n - i0, static_cast<uint64_t>(kAdamwBlock)));
      F2 m2[2], v2[2], root2[2], q2[2];
      if constexpr (BITS == 32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          m2[h] = pair(value<kF32, VEC>(in[b].m, 2 * h), value<kF32, VEC>(in[b].m, 2 * h + 1));
          v2[h] = pair(value<kF32, VEC>(in[b].v, 2 * h), value<kF32, VEC>(in[b].v, 2 * h + 1));
        }
      } else {
        decode4(in[b].mc, m2);
        decode4(in[b].vc, v2);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          m2[h] = mul2(m2[h], both(in[b].ms));
          v2[h] = mul2(v2[h], both(in[b].vs));
          v2[h] = mul2(v2[h], v2[h]);
        }
      }
      float m[kPer], v[kPer], root[kPer], den[kPer], quotient[kPer];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        F2 g = pair(value<GDT, VEC>(in[b].g, 2 * h), value<GDT, VEC>(in[b].g, 2 * h + 1));
        if (a.grad_scale != nullptr) g = mul2(g, both(grad_scale));
        m2[h] = add2(mul2(m2[h], both(a.beta1)), mul2(g, both(a.one_minus_beta1)), one);
        v2[h] = add2(mul2(v2[h], both(a.beta2)), mul2(mul2(g, g), both(a.one_minus_beta2)), one);
        root2[h] = sqrt2(v2[h]);
        const F2 d = add2(mul2(root2[h], both(a.root_scale)), both(a.eps), one);
        q2[h] = div2(m2[h], d);
        const float2 fm = parts(m2[h]), fv = parts(v2[h]), fr = parts(root2[h]), fq = parts(q2[h]);
        m[2 * h] = fm.x, m[2 * h + 1] = fm.y;
        v[2 * h] = fv.x, v[2 * h + 1] = fv.y;
        root[2 * h] = fr.x, root[2 * h + 1] = fr.y;
        quotient[2 * h] = fq.x, quotient[2 * h + 1] = fq.y;
      }
      // the ends of the exponent range: nonzero values below 2^-95, values
      // above 2^40, what is not finite
      uint32_t least = 0xFFFFFFFFu, top_m = 0, top_v = 0;
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        least = min(least, min(magnitude(m[q]) - 1, __float_as_uint(v[q]) - 1));
        top_m = max(top_m, magnitude(m[q]));
        top_v = max(top_v, __float_as_uint(v[q]));
      }
      const bool strange = a.any_range || least < kLeast - 1 || max(top_m, top_v) > kMost;
      if (__any_sync(0xFFFFFFFFu, strange)) {
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
          root[q] = __fsqrt_rn(v[q]);
          quotient[q] = __fdiv_rn(m[q], __fadd_rn(__fmul_rn(root[q], a.root_scale), a.eps));
        }
      }
      float p[kPer];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const F2 old = pair(value<PDT, VEC>(in[b].p, 2 * h), value<PDT, VEC>(in[b].p, 2 * h + 1));
        const float2 now = parts(add2(mul2(old, both(a.decay)),
                                      mul2(pair(quotient[2 * h], quotient[2 * h + 1]), both(-a.step_size)), one));
        p[2 * h] = now.x, p[2 * h + 1] = now.y;
      }
      store4<PDT, VEC>(t.param, i0, lane, count, p);
      if constexpr (COPY)
        if (t.copy != nullptr) store4<kBF16, VEC>(t.copy, i0, lane, count, p);
      if constexpr (BITS == 32) {
        store4<kF32, VEC>(t.m, i0, lane, count, m);
        store4<kF32, VEC>(t.v, i0, lane, count, v);
      } else {
        uint32_t top_root = 0;
#pragma unroll
        for (int q = 0; q < kPer; ++q) top_root = max(top_root, __float_as_uint(root[q]));
        top_m = __reduce_max_sync(0xFFFFFFFFu, top_m);
        top_root = __reduce_max_sync(0xFFFFFFFFu, top_root);
        const bool fine = max(top_m, top_root) < kInf;
        if (!fine) top_m = finite_top(m), top_root = finite_top(root);
        float mu, ms, vu, vs;
        block_scale(top_m, &mu, &ms);
        block_scale(top_root, &vu, &vs);
        uint32_t mc = 0, vc = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2 x = parts(mul2(pair(m[2 * h], m[2 * h + 1]), both(mu)));
          mc |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3)) << (16 * h);
        }
        if (vu > 0.0f) {  // else the block holds nothing worth a code
          const uint32_t threshold0 = static_cast<uint32_t>(i0 + element<VEC>(lane, 0)) * kDitherElem + a.dither;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // an e4m3 number times 2^-120 has its code in the top bits of its
            // fp32 form, subnormals included; the threshold below the last
            // code bit makes the carry that rounds up
            const float2 x = parts(mul2(mul2(pair(root[2 * h], root[2 * h + 1]), both(vu)), both(7.52316384526264e-37f)));
            const float xs[2] = {x.x, x.y};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int q = 2 * h + e;
              const uint32_t threshold = (threshold0 + static_cast<uint32_t>(VEC ? q : 32 * q) * kDitherElem) >> 12;
              const uint32_t low = v[q] > 0.0f ? 1u << 20 : 0u;  // a v that is not 0 has a code that is not 0
              const uint32_t bits = max(min(__float_as_uint(xs[e]), 0x7Eu << 20), low);
              vc |= (bits + threshold) >> 20 << (8 * q);
            }
          }
        }
        if (!fine) mc = mark_not_finite(mc, m), vc = mark_not_finite(vc, root);
        store_codes<VEC>(t.m, i0, lane, count, mc);
        store_codes<VEC>(t.v, i0, lane, count, vc);
        if (lane == 0) {
          t.m_scale[i0 / kAdamwBlock] = ms;
          t.v_scale[i0 / kAdamwBlock] = vs;
        }
      }
    }
  }
}

template <int PDT, int GDT, int BITS, bool COPY, typename Args>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Args a) {
  const int lane = threadIdx.x & 31;
  // the tensor of this chunk: the last whose first chunk is not past it
  int at = -1;
  for (int i = 0; i < a.count; i += 32)
    at += __popc(__ballot_sync(0xFFFFFFFFu, i + lane < a.count && a.chunk0[min(i + lane, a.count)] <= blockIdx.x));
  const AdamwTensor& t = a.t[at];
  const uint64_t c0 = static_cast<uint64_t>(blockIdx.x - a.chunk0[at]) * kAdamwChunk;
  uintptr_t off = (reinterpret_cast<uintptr_t>(t.param) & (PDT == kF32 ? 15 : 7)) |
                  (reinterpret_cast<uintptr_t>(t.grad) & (GDT == kF32 ? 15 : 7)) |
                  ((reinterpret_cast<uintptr_t>(t.m) | reinterpret_cast<uintptr_t>(t.v)) & (BITS == 32 ? 15 : 3));
  if (COPY) off |= reinterpret_cast<uintptr_t>(t.copy) & 7;
  pdl_enter();
  const float grad_scale = a.grad_scale != nullptr ? *a.grad_scale : 1.0f;
  if (off == 0) adamw_chunk<PDT, GDT, BITS, COPY, true>(a, t, c0, grad_scale);
  else adamw_chunk<PDT, GDT, BITS, COPY, false>(a, t, c0, grad_scale);
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
