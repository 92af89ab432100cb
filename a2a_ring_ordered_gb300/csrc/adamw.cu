// adamw.cu -- one AdamW step over many tensors, states in 32 or 8 bits.
//
// Per element (include/ccl.h has the formula): read the parameter, its
// gradient and two moments, write the parameter and the moments, every
// operation rounded to fp32 by itself so that the result does not depend on
// how the compiler contracts it.  Bound by HBM: 26 bytes per element with
// fp32 parameters and states and bf16 gradients, 14.125 with 8-bit states (and
// 2 for a bf16 copy).  Measured with the copy, 157 M elements: fp32 states 629
// us (7.0 TB/s); 8-bit states 429 us (5.9 TB/s) with every array on the
// vectors' grid, where issue slots (0.71 a cycle) and HBM are both two thirds
// full; 480 with parameters, gradients and copies off it: a tenth more
// instructions, for which the stage's vectors cannot serve, since stores of
// neighbours per lane would ask for every sector four times.  Without a copy:
// fp32 gradients 412 us, off the grid 457; bf16 parameters and gradients 395 and
// 459, bound by the same instructions for 10 bytes an element.
//
// An 8-bit state is e4m3 codes with one fp32 scale per 128 elements.  A warp
// holds such a block with four elements per lane, so its amax is one
// warp-wide integer maximum of the magnitudes' bits.
#include <cuda_fp8.h>

#include <atomic>

#include "device_common.cuh"

namespace ccl {
namespace {

constexpr int kPer = 4;  // elements per lane: a warp holds a block of 128
constexpr int kBlocksPerWarp = kAdamwChunk / kAdamwBlock / (kThreads / 32);
constexpr uint32_t kDitherElem = 1779033703u;
constexpr uint32_t kInf = 0x7F800000u;

// ------------------------------------------------------- elements of a lane
// VEC: lane l holds elements 4 l .. 4 l + 3 of a block, by one vector access
// (every array of the tensor on the vector's grid, the block whole).
// Otherwise elements l, l + 32, l + 64, l + 96, so that each of the four
// accesses of a warp is one contiguous run wherever the array starts; with
// four neighbours per lane the scalar accesses of an array off the grid asked
// L2 for every sector four times (157 M elements with 8-bit states 869 us
// against 696 on the grid).  WHOLE: the block has all of its 128 elements.
template <bool VEC>
__device__ __forceinline__ int element(int lane, int q) {
  return VEC ? lane * kPer + q : lane + 32 * q;
}

// Parameters and moments are written by this kernel: no read-only path, and
// in the program's order before the stores.
__device__ __forceinline__ uint4 ld_own16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_own8(const void* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld_own4(const void* p) {
  uint32_t v;
  asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld_own2(const void* p) {
  unsigned short v;
  asm volatile("ld.global.L1::no_allocate.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}

template <int DT>
struct Raw4 {
  uint32_t w[kPer];  // VEC: as loaded; else element q in the low bits of w[q]
};
// The lane's elements of the block at `base` + i0, which has `count` elements; zeros behind them.
template <int DT, bool VEC, bool WHOLE>
__device__ __forceinline__ void load4(const void* base, uint64_t i0, int lane, int count, Raw4<DT>& r) {
  const char* p = static_cast<const char*>(base) + i0 * Elem<DT>::kBytes;
  if constexpr (VEC && DT == kF32) {
    const uint4 v = ld_own16(p + lane * 16);
    r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
  } else if constexpr (VEC) {
    const uint2 v = ld_own8(p + lane * 8);
    r.w[0] = v.x, r.w[1] = v.y;
  } else {
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int i = element<VEC>(lane, q);
      r.w[q] = !WHOLE && i >= count ? 0u : DT == kF32 ? ld_own4(p + i * 4) : ld_own2(p + i * 2);
    }
  }
}
template <int DT, bool VEC>
__device__ __forceinline__ float value(const Raw4<DT>& r, int q) {
  if constexpr (VEC || DT == kF32) return widen<DT>(r.w, q);
  else return __uint_as_float(r.w[q] << 16);
}
template <int DT, bool VEC, bool WHOLE>
__device__ __forceinline__ void store4(void* base, uint64_t i0, int lane, int count, const float* x) {
  char* p = static_cast<char*>(base) + i0 * Elem<DT>::kBytes;
  uint32_t w[kPer];
  if constexpr (VEC) {
    pack_out<DT, kPer>(x, w);
    if constexpr (DT == kF32) st_stream16(p + lane * 16, make_uint4(w[0], w[1], w[2], w[3]));
    else __stcs(reinterpret_cast<uint2*>(p + lane * 8), make_uint2(w[0], w[1]));
  } else {
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int i = element<VEC>(lane, q);
      if (!WHOLE && i >= count) continue;
      pack_out<DT, 1>(x + q, w);
      store_one<DT>(p, i, w, 0);
    }
  }
}
template <bool VEC, bool WHOLE>
__device__ __forceinline__ void store_codes(void* base, uint64_t i0, int lane, int count, uint32_t w) {
  uint8_t* p = static_cast<uint8_t*>(base) + i0;
  if constexpr (VEC) {
    st_stream4(p + lane * kPer, w);
  } else {
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int i = element<VEC>(lane, q);
      if (WHOLE || i < count) __stcs(p + i, static_cast<uint8_t>(w >> (8 * q)));
    }
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
__device__ __forceinline__ F2 both(const AdamwPair& c) { return F2{c.v}; }
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
__device__ __forceinline__ F2 sqrt2(F2 x, const AdamwPairs& k) {
  const float2 s = parts(x);
  const F2 y = pair(s.x > 0.0f ? rsqrt_approx(s.x) : 0.0f, s.y > 0.0f ? rsqrt_approx(s.y) : 0.0f);
  F2 g = mul2(x, y), nh = mul2(y, both(k.minus_half));  // sqrt(x) and -1 / (2 sqrt(x)), nearly
  const F2 r = fma2(nh, g, both(k.half));
  g = fma2(g, r, g);
  nh = fma2(nh, r, nh);
  const F2 d = fma2(g, g, mul2(x, both(k.minus_one)));  // g^2 - x, exact
  return fma2(nh, d, g);
}
__device__ __forceinline__ F2 div2(F2 a, F2 b, const AdamwPairs& k) {
  const float2 s = parts(b);
  F2 y = pair(rcp_approx(s.x), rcp_approx(s.y));
  const F2 nb = mul2(b, both(k.minus_one));
  y = fma2(fma2(nb, y, both(k.one)), y, y);
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
// are made with, and the scale.  The reciprocal is rounded to nearest, by one
// correction as in div2 while amax is at most 2^40.
__device__ __forceinline__ void block_scale(uint32_t top, float* up, float* scale) {
  const float amax = __uint_as_float(top);
  const bool some = amax > 7.888609052210118e-31f;  // 2^-100
  float y = rcp_approx(amax);
  y = fmaf(fmaf(-amax, y, 1.0f), y, y);
  if (top > kMost) y = __frcp_rn(amax);
  *up = some ? __fmul_rn(y, 448.0f) : 0.0f;
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

constexpr int kTogether = 2;  // blocks that a warp works on at a time: a factor that has been fetched serves both

// The step on two blocks whose inputs are in registers.
template <int PDT, int GDT, int BITS, bool COPY, bool VEC, bool WHOLE, typename Args>
__device__ __forceinline__ void adamw_blocks(const Args& a, const AdamwTensor& t, const uint64_t* i0, const int* count,
                                             const Inputs<PDT, GDT, BITS>* in, float grad_scale) {
  constexpr int U = kTogether, kPairs = U * kPer / 2;  // pairs of elements: two per block
  const int lane = threadIdx.x & 31;
  const F2 one = both(a.k.one);
  F2 m2[kPairs], v2[kPairs], root2[kPairs], q2[kPairs];
#pragma unroll
  for (int b = 0; b < U; ++b) {
    if constexpr (BITS == 8) {
      decode4(in[b].mc, m2 + 2 * b);
      decode4(in[b].vc, v2 + 2 * b);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = 2 * b + h;
      if constexpr (BITS == 32) {
        m2[k] = pair(value<kF32, VEC>(in[b].m, 2 * h), value<kF32, VEC>(in[b].m, 2 * h + 1));
        v2[k] = pair(value<kF32, VEC>(in[b].v, 2 * h), value<kF32, VEC>(in[b].v, 2 * h + 1));
      } else {
        m2[k] = mul2(m2[k], both(in[b].ms));
        v2[k] = mul2(v2[k], both(in[b].vs));
        v2[k] = mul2(v2[k], v2[k]);
      }
      F2 g = pair(value<GDT, VEC>(in[b].g, 2 * h), value<GDT, VEC>(in[b].g, 2 * h + 1));
      if (a.grad_scale != nullptr) g = mul2(g, both(grad_scale));
      m2[k] = add2(mul2(m2[k], both(a.k.beta1)), mul2(g, both(a.k.one_minus_beta1)), one);
      v2[k] = add2(mul2(v2[k], both(a.k.beta2)), mul2(mul2(g, g), both(a.k.one_minus_beta2)), one);
    }
  }
#pragma unroll
  for (int k = 0; k < kPairs; ++k) root2[k] = sqrt2(v2[k], a.k);
#pragma unroll
  for (int k = 0; k < kPairs; ++k)
    q2[k] = div2(m2[k], add2(mul2(root2[k], both(a.k.root_scale)), both(a.k.eps), one), a.k);
  // the ends of the exponent range: nonzero values below 2^-95, values
  // above 2^40, what is not finite
  uint32_t least = 0xFFFFFFFFu, top_m[U] = {}, top_v = 0;
#pragma unroll
  for (int k = 0; k < kPairs; ++k) {
    const float2 fm = parts(m2[k]), fv = parts(v2[k]);
    least = min(min(least, min(magnitude(fm.x) - 1, magnitude(fm.y) - 1)), min(__float_as_uint(fv.x) - 1, __float_as_uint(fv.y) - 1));
    top_m[k >> 1] = max(top_m[k >> 1], max(magnitude(fm.x), magnitude(fm.y)));
    top_v = max(top_v, max(__float_as_uint(fv.x), __float_as_uint(fv.y)));
  }
  const bool strange = a.any_range || least < kLeast - 1 || max(max(top_m[0], top_m[U - 1]), top_v) > kMost;
  const bool exact = __any_sync(0xFFFFFFFFu, strange);
  if (exact) {
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      const float2 fm = parts(m2[k]), fv = parts(v2[k]);
      const float r0 = __fsqrt_rn(fv.x), r1 = __fsqrt_rn(fv.y);
      root2[k] = pair(r0, r1);
      q2[k] = pair(__fdiv_rn(fm.x, __fadd_rn(__fmul_rn(r0, a.root_scale), a.eps)),
                   __fdiv_rn(fm.y, __fadd_rn(__fmul_rn(r1, a.root_scale), a.eps)));
    }
  }
#pragma unroll
  for (int b = 0; b < U; ++b) {
    if (!WHOLE && count[b] == 0) return;
    float p[kPer], m[kPer], v[kPer], root[kPer];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = 2 * b + h;
      const F2 old = pair(value<PDT, VEC>(in[b].p, 2 * h), value<PDT, VEC>(in[b].p, 2 * h + 1));
      const float2 now = parts(add2(mul2(old, both(a.k.decay)), mul2(q2[k], both(a.k.minus_step)), one));
      const float2 fm = parts(m2[k]), fv = parts(v2[k]), fr = parts(root2[k]);
      p[2 * h] = now.x, p[2 * h + 1] = now.y;
      m[2 * h] = fm.x, m[2 * h + 1] = fm.y;
      v[2 * h] = fv.x, v[2 * h + 1] = fv.y;
      root[2 * h] = fr.x, root[2 * h + 1] = fr.y;
    }
    store4<PDT, VEC, WHOLE>(t.param, i0[b], lane, count[b], p);
    if constexpr (COPY)
      if (t.copy != nullptr) store4<kBF16, VEC, WHOLE>(t.copy, i0[b], lane, count[b], p);
    if constexpr (BITS == 32) {
      store4<kF32, VEC, WHOLE>(t.m, i0[b], lane, count[b], m);
      store4<kF32, VEC, WHOLE>(t.v, i0[b], lane, count[b], v);
    } else {
      uint32_t top_root = 0;
#pragma unroll
      for (int q = 0; q < kPer; ++q) top_root = max(top_root, __float_as_uint(root[q]));
      uint32_t tm = __reduce_max_sync(0xFFFFFFFFu, top_m[b]);
      top_root = __reduce_max_sync(0xFFFFFFFFu, top_root);
      const bool fine = !exact || max(tm, top_root) < kInf;
      if (!fine) tm = finite_top(m), top_root = finite_top(root);
      float mu, ms, vu, vs;
      block_scale(tm, &mu, &ms);
      block_scale(top_root, &vu, &vs);
      uint32_t mc = 0, vc = 0;
      const uint32_t threshold0 = static_cast<uint32_t>(i0[b] + element<VEC>(lane, 0)) * kDitherElem + a.dither;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = 2 * b + h;
        const float2 x = parts(mul2(m2[k], both(mu)));
        mc |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3)) << (16 * h);
        // an e4m3 number times 2^-120 has its code in the top bits of its
        // fp32 form, subnormals included; the threshold below the last code
        // bit makes the carry that rounds up
        const float2 y = parts(mul2(mul2(root2[k], both(vu)), both(a.k.tiny)));
        const float ys[2] = {y.x, y.y};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int q = 2 * h + e;
          const uint32_t threshold = (threshold0 + static_cast<uint32_t>(VEC ? q : 32 * q) * kDitherElem) >> 12;
          const uint32_t low = min(__float_as_uint(root[q]), 1u << 20);  // a v that is not 0 has a code that is not 0
          const uint32_t bits = max(min(__float_as_uint(ys[e]), 0x7Eu << 20), low);
          vc |= (bits + threshold) >> 20 << (8 * q);
        }
      }
      if (!(vu > 0.0f)) vc = 0;  // the block holds nothing worth a code
      if (!fine) mc = mark_not_finite(mc, m), vc = mark_not_finite(vc, root);
      store_codes<VEC, WHOLE>(t.m, i0[b], lane, count[b], mc);
      store_codes<VEC, WHOLE>(t.v, i0[b], lane, count[b], vc);
      if (lane == 0) {
        t.m_scale[i0[b] / kAdamwBlock] = ms;
        t.v_scale[i0[b] / kAdamwBlock] = vs;
      }
    }
  }
}

// ------------------------------------------------- fp32 states: registers
// A chunk of one tensor: warp w takes blocks w, w + 8, ..., two at a time,
// whose loads are on the way together.
template <int PDT, int GDT, bool COPY, bool VEC, bool WHOLE, typename Args>
__device__ __forceinline__ void adamw_chunk(const Args& a, const AdamwTensor& t, uint64_t c0, float grad_scale) {
  static_assert(kBlocksPerWarp % kTogether == 0, "whole batches");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll 1
  for (int b0 = 0; b0 < kBlocksPerWarp; b0 += kTogether) {
    uint64_t i0[kTogether];
    int count[kTogether];  // elements of the block
    Inputs<PDT, GDT, 32> in[kTogether];
#pragma unroll
    for (int b = 0; b < kTogether; ++b) {
      i0[b] = c0 + static_cast<uint64_t>((b0 + b) * (kThreads / 32) + warp) * kAdamwBlock;
      count[b] = WHOLE ? kAdamwBlock : static_cast<int>(min(t.n - min(i0[b], t.n), static_cast<uint64_t>(kAdamwBlock)));
      if (!WHOLE && count[0] == 0) return;  // the whole warp
      load4<PDT, VEC, WHOLE>(t.param, i0[b], lane, count[b], in[b].p);
      load4<GDT, VEC, WHOLE>(t.grad, i0[b], lane, count[b], in[b].g);
      load4<kF32, VEC, WHOLE>(t.m, i0[b], lane, count[b], in[b].m);
      load4<kF32, VEC, WHOLE>(t.v, i0[b], lane, count[b], in[b].v);
    }
    adamw_blocks<PDT, GDT, 32, COPY, VEC, WHOLE>(a, t, i0, count, in, grad_scale);
  }
}

// The tensor of a chunk: the last whose first chunk is not past it.
template <typename Args>
__device__ __forceinline__ int tensor_of(const Args& a, uint32_t chunk) {
  const int lane = threadIdx.x & 31;
  int at = -1;
  for (int i = 0; i < a.count; i += 32)
    at += __popc(__ballot_sync(0xFFFFFFFFu, i + lane < a.count && a.chunk0[min(i + lane, a.count)] <= chunk));
  return __shfl_sync(0xFFFFFFFFu, at, 0);  // the same in every lane, and known to be
}

// Whether every array of the tensor is on the grid of a lane's vector.
template <int PDT, int GDT, int BITS>
__device__ __forceinline__ bool on_vectors(const AdamwTensor& t) {
  return ((reinterpret_cast<uintptr_t>(t.param) & (PDT == kF32 ? 15 : 7)) | (reinterpret_cast<uintptr_t>(t.grad) & (GDT == kF32 ? 15 : 7)) |
          ((reinterpret_cast<uintptr_t>(t.m) | reinterpret_cast<uintptr_t>(t.v)) & (BITS == 32 ? 15 : 3)) |
          (reinterpret_cast<uintptr_t>(t.copy) & 7)) == 0;
}

template <int PDT, int GDT, bool COPY, typename Args>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Args a) {
  const int at = tensor_of(a, blockIdx.x);
  const AdamwTensor& t = a.t[at];
  const uint64_t c0 = static_cast<uint64_t>(blockIdx.x - a.chunk0[at]) * kAdamwChunk;
  pdl_enter();
  const float grad_scale = a.grad_scale != nullptr ? *a.grad_scale : 1.0f;
  const bool whole = c0 + kAdamwChunk <= t.n;
  if (whole && on_vectors<PDT, GDT, 32>(t)) adamw_chunk<PDT, GDT, COPY, true, true>(a, t, c0, grad_scale);
  else if (whole) adamw_chunk<PDT, GDT, COPY, false, true>(a, t, c0, grad_scale);
  else adamw_chunk<PDT, GDT, COPY, false, false>(a, t, c0, grad_scale);
}

// ---------------------------------------------- 8-bit states: a copied stage
// With 8-bit states a block takes half the bytes and twice the arithmetic of
// one with fp32 states: loads into registers then hold a warp up for as long
// as its arithmetic does (157 M elements 622 us).  So a ninth warp of a
// persistent CTA has the next chunk's arrays copied into shared memory while
// the others work on one; the copies are whole 16-byte granules, which fits
// every alignment.  The warps wait for the copies and give the stage back each
// by itself (with barriers of the whole CTA in their place, and every warp
// looking the tensor up: 553 us).
constexpr int kStreamStages = 2;
constexpr long long kWaitCycles = 1ll << 32;  // two seconds

__device__ unsigned int g_adamw_error;  // nonzero: a bounded wait ran out
std::atomic<bool> g_streamed{false};    // whether a kernel that waits was launched; never taken back

template <int PDT, int GDT>
struct alignas(16) Stage {
  char p[kAdamwChunk * Elem<PDT>::kBytes + 16];
  char g[kAdamwChunk * Elem<GDT>::kBytes + 16];
  char m[kAdamwChunk + 16], v[kAdamwChunk + 16];
  char ms[kAdamwChunk / kAdamwBlock * 4 + 16], vs[kAdamwChunk / kAdamwBlock * 4 + 16];
};
template <int PDT, int GDT>
struct StreamShared {
  Stage<PDT, GDT> stage[kStreamStages];
  AdamwTensor tensor[kStreamStages];  // of the chunk in the stage
  uint64_t c0[kStreamStages];         // and its first element
  uint64_t full[kStreamStages], empty[kStreamStages];
  uint32_t dead;  // a wait ran out
};
constexpr int kStreamThreads = kThreads + 32;
// CTAs that an SM's 228 KB hold, 1 KB of each the system's, three at most: two
// where parameters and gradients are fp32 (82 KB a CTA).  Chunks are dealt out by
// the grid, so it may not have more CTAs than run together.
template <int PDT, int GDT>
constexpr int kCtasPerSm = (228 << 10) / (sizeof(StreamShared<PDT, GDT>) + 1024) < 3 ? (228 << 10) / (sizeof(StreamShared<PDT, GDT>) + 1024) : 3;

__device__ __forceinline__ uint32_t shared_address(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// Copies the granules of `bytes` bytes at src to dst; returns the bytes on the way.
__device__ __forceinline__ uint32_t copy_granules(char* dst, const void* src, uint32_t bytes, uint32_t bar) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(src) & ~static_cast<uintptr_t>(15);
  const uint32_t size = static_cast<uint32_t>(((reinterpret_cast<uintptr_t>(src) + bytes + 15) & ~static_cast<uintptr_t>(15)) - lo);
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(shared_address(dst)),
               "l"(lo), "r"(size), "r"(bar)
               : "memory");
  return size;
}
__device__ __forceinline__ uint32_t granule_bytes(const void* src, uint32_t bytes) {
  return static_cast<uint32_t>(((reinterpret_cast<uintptr_t>(src) + bytes + 15) & ~static_cast<uintptr_t>(15)) -
                               (reinterpret_cast<uintptr_t>(src) & ~static_cast<uintptr_t>(15)));
}
// Where the bytes of src begin in the stage.
__device__ __forceinline__ const char* staged(const char* stage, const void* src) {
  return stage + (reinterpret_cast<uintptr_t>(src) & 15);
}

template <int PDT, int GDT>
__device__ __forceinline__ void copy_chunk(const AdamwTensor& t, uint64_t c0, Stage<PDT, GDT>& s, uint32_t bar) {
  const uint32_t n = static_cast<uint32_t>(min(t.n - c0, static_cast<uint64_t>(kAdamwChunk)));
  const uint32_t scales = (n + kAdamwBlock - 1) / kAdamwBlock * 4;
  const char* p = static_cast<const char*>(t.param) + c0 * Elem<PDT>::kBytes;
  const char* g = static_cast<const char*>(t.grad) + c0 * Elem<GDT>::kBytes;
  const char *m = static_cast<const char*>(t.m) + c0, *v = static_cast<const char*>(t.v) + c0;
  const float *ms = t.m_scale + c0 / kAdamwBlock, *vs = t.v_scale + c0 / kAdamwBlock;
  const uint32_t bytes = granule_bytes(p, n * Elem<PDT>::kBytes) + granule_bytes(g, n * Elem<GDT>::kBytes) + granule_bytes(m, n) +
                         granule_bytes(v, n) + granule_bytes(ms, scales) + granule_bytes(vs, scales);
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
  copy_granules(s.p, p, n * Elem<PDT>::kBytes, bar);
  copy_granules(s.g, g, n * Elem<GDT>::kBytes, bar);
  copy_granules(s.m, m, n, bar);
  copy_granules(s.v, v, n, bar);
  copy_granules(s.ms, ms, scales, bar);
  copy_granules(s.vs, vs, scales, bar);
}

template <int DT, bool VEC>
__device__ __forceinline__ void take4(const char* base, int i0, int lane, Raw4<DT>& r) {
  const char* p = base + i0 * Elem<DT>::kBytes;
  if constexpr (VEC && DT == kF32) {
    const uint4 v = *reinterpret_cast<const uint4*>(p + lane * 16);
    r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
  } else if constexpr (VEC) {
    const uint2 v = *reinterpret_cast<const uint2*>(p + lane * 8);
    r.w[0] = v.x, r.w[1] = v.y;
  } else {
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      if constexpr (DT == kF32) r.w[q] = *reinterpret_cast<const uint32_t*>(p + 4 * (lane + 32 * q));
      else r.w[q] = *reinterpret_cast<const uint16_t*>(p + 2 * (lane + 32 * q));
    }
  }
}
template <bool VEC>
__device__ __forceinline__ uint32_t take_codes(const char* base, int i0, int lane) {
  const uint8_t* p = reinterpret_cast<const uint8_t*>(base) + i0;
  if constexpr (VEC) return *reinterpret_cast<const uint32_t*>(p + 4 * lane);
  return p[lane] | p[lane + 32] << 8 | p[lane + 64] << 16 | static_cast<uint32_t>(p[lane + 96]) << 24;
}

template <int PDT, int GDT, bool COPY, bool VEC, bool WHOLE, typename Args>
__device__ __forceinline__ void staged_chunk(const Args& a, const AdamwTensor& t, uint64_t c0, const Stage<PDT, GDT>& s, float grad_scale) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const char* p = staged(s.p, static_cast<const char*>(t.param) + c0 * Elem<PDT>::kBytes);
  const char* g = staged(s.g, static_cast<const char*>(t.grad) + c0 * Elem<GDT>::kBytes);
  const char *m = staged(s.m, static_cast<const char*>(t.m) + c0), *v = staged(s.v, static_cast<const char*>(t.v) + c0);
  const float* ms = reinterpret_cast<const float*>(staged(s.ms, t.m_scale + c0 / kAdamwBlock));
  const float* vs = reinterpret_cast<const float*>(staged(s.vs, t.v_scale + c0 / kAdamwBlock));
#pragma unroll 1
  for (int b0 = 0; b0 < kBlocksPerWarp; b0 += kTogether) {
    uint64_t i0[kTogether];
    int count[kTogether];
    Inputs<PDT, GDT, 8> in[kTogether];
#pragma unroll
    for (int b = 0; b < kTogether; ++b) {
      const int block = (b0 + b) * (kThreads / 32) + warp;
      i0[b] = c0 + static_cast<uint64_t>(block) * kAdamwBlock;
      count[b] = WHOLE ? kAdamwBlock : static_cast<int>(min(t.n - min(i0[b], t.n), static_cast<uint64_t>(kAdamwBlock)));
      if (!WHOLE && count[0] == 0) return;  // the whole warp
      take4<PDT, VEC>(p, block * kAdamwBlock, lane, in[b].p);
      take4<GDT, VEC>(g, block * kAdamwBlock, lane, in[b].g);
      in[b].mc = take_codes<VEC>(m, block * kAdamwBlock, lane);
      in[b].vc = take_codes<VEC>(v, block * kAdamwBlock, lane);
      in[b].ms = ms[block];
      in[b].vs = vs[block];
      if (!WHOLE) {  // what lies behind the tensor's end is not of it
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
          if (element<VEC>(lane, q) < count[b]) continue;
          in[b].p.w[q] = in[b].g.w[q] = 0;
          in[b].mc &= ~(0xFFu << (8 * q));
          in[b].vc &= ~(0xFFu << (8 * q));
        }
        if (count[b] == 0) in[b].ms = in[b].vs = 1.0f;
      }
    }
    adamw_blocks<PDT, GDT, 8, COPY, VEC, WHOLE>(a, t, i0, count, in, grad_scale);
  }
}

// Waits for a barrier's phase; false once this or another wait of the CTA ran out.
__device__ __forceinline__ bool stream_wait(uint64_t* barrier, uint32_t parity, volatile uint32_t* dead, long long cycles = kWaitCycles) {
  const uint32_t bar = shared_address(barrier);
  const long long t0 = clock64();
  for (;;) {
    uint32_t done;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(done)
                 : "r"(bar), "r"(parity)
                 : "memory");
    if (done) return true;
    if (*dead) return false;
    if (clock64() - t0 > cycles) {
      *dead = 1;
      atomicExch(&g_adamw_error, kAdamwError);
      return false;
    }
  }
}

template <int PDT, int GDT, bool COPY, typename Args>
__global__ void __launch_bounds__(kStreamThreads, kCtasPerSm<PDT, GDT>) adamw_stream_kernel(const __grid_constant__ Args a) {
  extern __shared__ char raw[];
  StreamShared<PDT, GDT>& s = *reinterpret_cast<StreamShared<PDT, GDT>*>(raw);
  const uint32_t chunks = a.chunk0[a.count];
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStreamStages; ++i) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(shared_address(&s.full[i])) : "memory");
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(shared_address(&s.empty[i])), "r"(kThreads / 32) : "memory");
    }
    s.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  pdl_enter();
  uint32_t st = 0, phase = 0;
  if (threadIdx.x >= kThreads) {  // the copying warp
    bool ok = true;
    for (uint32_t chunk = blockIdx.x; ok && chunk < chunks; chunk += gridDim.x) {
      const int at = tensor_of(a, chunk);
      if (lane == 0) {
        ok = stream_wait(&s.empty[st], phase ^ 1, &s.dead);
        if (ok) {
          const AdamwTensor& t = a.t[at];
          const uint64_t c0 = static_cast<uint64_t>(chunk - a.chunk0[at]) * kAdamwChunk;
          s.tensor[st] = t;
          s.c0[st] = c0;
          copy_chunk<PDT, GDT>(t, c0, s.stage[st], shared_address(&s.full[st]));
        }
      }
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      if (++st == kStreamStages) st = 0, phase ^= 1;
    }
    // every stage given back: no copy is on its way to a CTA that has left, not
    // even where the others' wait for it ran out
    for (int j = 0; ok && j < kStreamStages; ++j) {
      if (lane == 0) ok = stream_wait(&s.empty[st], phase ^ 1, &s.dead);
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      if (++st == kStreamStages) st = 0, phase ^= 1;
    }
    if (!ok) {  // copies in flight still write this CTA's shared memory
      const long long t1 = clock64();
      while (clock64() - t1 < (1ll << 22)) {
      }
    }
    return;
  }
  const float grad_scale = a.grad_scale != nullptr ? *a.grad_scale : 1.0f;
  for (uint32_t chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x) {
    if (!__all_sync(0xFFFFFFFFu, stream_wait(&s.full[st], phase, &s.dead))) return;
    const AdamwTensor t = s.tensor[st];
    const uint64_t c0 = s.c0[st];
    const bool whole = c0 + kAdamwChunk <= t.n;
    if (whole && on_vectors<PDT, GDT, 8>(t)) staged_chunk<PDT, GDT, COPY, true, true>(a, t, c0, s.stage[st], grad_scale);
    else if (whole) staged_chunk<PDT, GDT, COPY, false, true>(a, t, c0, s.stage[st], grad_scale);
    else staged_chunk<PDT, GDT, COPY, false, false>(a, t, c0, s.stage[st], grad_scale);
    __syncwarp();
    if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(shared_address(&s.empty[st])) : "memory");
    if (++st == kStreamStages) st = 0, phase ^= 1;
  }
}

// Self-test of the bounded wait: a barrier that nothing completes.
__global__ void __launch_bounds__(32) adamw_wait_probe_kernel(long long cycles) {
  __shared__ alignas(8) uint64_t bar;
  __shared__ uint32_t dead;
  if (threadIdx.x != 0) return;
  dead = 0;
  asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(shared_address(&bar)) : "memory");
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  stream_wait(&bar, 0, &dead, cycles);
}

template <int PDT, int GDT, int BITS, bool COPY, typename Args>
cudaError_t launch_one(const Args& a, cudaStream_t s) {
  if constexpr (BITS == 32) {
    return launch_kernel(adamw_kernel<PDT, GDT, COPY, Args>, dim3(a.chunk0[a.count]), dim3(kThreads), s, a);
  } else {
    constexpr size_t smem = sizeof(StreamShared<PDT, GDT>);
    static_assert(kCtasPerSm<PDT, GDT> >= 1 && kCtasPerSm<PDT, GDT> * (smem + 1024) <= 228 << 10, "every CTA of the grid runs at once");
    const auto kernel = adamw_stream_kernel<PDT, GDT, COPY, Args>;
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (err != cudaSuccess) return err;
    const uint32_t resident = static_cast<uint32_t>(current_sm_count()) * kCtasPerSm<PDT, GDT>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.chunk0[a.count] < resident || resident == 0 ? a.chunk0[a.count] : resident);
    cfg.blockDim = dim3(kStreamThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = CCL_PDL ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    g_streamed.store(true, std::memory_order_relaxed);
    return cudaLaunchKernelEx(&cfg, kernel, a);
  }
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

cudaError_t launch_adamw_wait_probe(cudaStream_t s) {
  g_streamed.store(true, std::memory_order_relaxed);
  adamw_wait_probe_kernel<<<1, 32, 0, s>>>(1ll << 14);
  const cudaError_t err = cudaGetLastError();
  if (err == cudaSuccess) note_launch();
  return err;
}

cudaError_t read_adamw_error(unsigned int* flag, bool clear) {
  *flag = 0;
  if (!g_streamed.load(std::memory_order_relaxed)) return cudaSuccess;
  cudaError_t err = cudaMemcpyFromSymbol(flag, g_adamw_error, sizeof(unsigned int));
  if (err == cudaSuccess && clear && *flag != 0) {
    const unsigned int zero = 0;
    err = cudaMemcpyToSymbol(g_adamw_error, &zero, sizeof(zero));
  }
  return err;
}

cudaError_t launch_adamw(int param_dt, int grad_dt, int bits, bool copy, const AdamwSmall& a, cudaStream_t s) {
  return launch_any(param_dt, grad_dt, bits, copy, a, s);
}
cudaError_t launch_adamw(int param_dt, int grad_dt, int bits, bool copy, const AdamwLarge& a, cudaStream_t s) {
  return launch_any(param_dt, grad_dt, bits, copy, a, s);
}

}  // namespace ccl
