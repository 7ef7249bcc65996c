// fp4.cuh -- the blocked scale layout and element conversions of the microscaled 4-bit
// formats, shared by the encoder / decoder (fp4.cu) and the product (fp4_gemm.cu).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "mxfp4.cuh"

namespace csa {

__host__ __device__ constexpr int fp4_block(bool nv) { return nv ? 16 : 32; }  // elements per scale

// scale atoms (128 rows x 4 scales, 512 bytes) along a row of `cols` elements
__host__ __device__ constexpr int fp4_atoms(bool nv, int cols) {
  return (cols + 4 * fp4_block(nv) - 1) / (4 * fp4_block(nv));
}

// byte offset of the atom (row block, atom) of a matrix with n_atoms per row block
__host__ __device__ constexpr int64_t fp4_atom_offset(int64_t row_block, int atom, int n_atoms) {
  return (row_block * n_atoms + atom) * 512;
}

__device__ __forceinline__ float e4m3_value(uint32_t byte) {  // exact; 0x7F / 0xFF are NaN
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3)));
}

// x / T correctly rounded, given r = 1 / T correctly rounded, for |x| <= 8 T and T in
// [2^-90, 2^100]: two residual steps (P. Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990).  q0 is within 1.5 units in the last place, q1 within one,
// and a residual step from a quotient within one unit, with a correctly rounded reciprocal, rounds
// correctly.  Residuals of an x too small for an exact one only meet quotients that encode as 0.
// The residual is taken as q T - x, so that a zero keeps its sign.
__device__ __forceinline__ float div_given_rcp(float x, float T, float r) {
  const float q0 = x * r;
  const float q1 = fmaf(-fmaf(q0, T, -x), r, q0);
  return fmaf(-fmaf(q1, T, -x), r, q1);
}

// four quotients by plain division, zeros for T = 0 (out of line: unrolled, they would crowd the
// instruction cache of every kernel that encodes, and only blocks with an extreme scale come here)
static __device__ __noinline__ float4 div4(float a, float b, float c, float d, float T) {
  if (T == 0.f) return make_float4(0.f, 0.f, 0.f, 0.f);
  return make_float4(__fdiv_rn(a, T), __fdiv_rn(b, T), __fdiv_rn(c, T), __fdiv_rn(d, T));
}

// The range of divisors that div_given_rcp takes.
__device__ __forceinline__ bool div_range(float T) { return T >= 0x1p-90f && T <= 0x1p100f; }

// Whether a block's quotients take plain division: a scale cut at 448, a T out of range, or (bf16 values)
// one whose significand is all ones (see nv_codes8_common).
template <bool kBf16>
__device__ __forceinline__ bool nv_plain(float T, float amax) {
  return !(div_range(T) && amax <= 8.f * T) || (kBf16 && (__float_as_uint(T) & 0x7FFFFFu) == 0x7FFFFFu);
}

// NVFP4's encoder constants of a tensor: its scale g, and 6 g with the reciprocal.
struct NvScale {
  float g, six_g, rcp;
  __device__ __forceinline__ explicit NvScale(float scale) {
    g = scale;
    six_g = 6.f * scale;
    rcp = __frcp_rn(six_g);
  }
  // scale byte of a block: e4m3(amax / (6 g)), to nearest even, at most 448 (amax is cut at 1024 times
  // 6 g, far beyond; quotients too small for an exact residual are 0 in e4m3 anyway); 0 / 0, a block of zeros
  // under g = 0 (which a tensor of zeros has for its largest value / 2688), counts as 0
  __device__ __forceinline__ uint32_t byte(float amax) const {
    const float q = div_range(six_g) ? div_given_rcp(fminf(amax, 1024.f * six_g), six_g, rcp)
                                     : fmaxf(__fdiv_rn(amax, six_g), 0.f);
    return __nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
  }
};

// The quotients x / T of kN values of a block under its NVFP4 scale T (zeros if T is zero).
// amax: the block's; where its scale is cut at 448 or T is extreme, plain division, after the
// common case so that several blocks' arithmetic can overlap.
template <int kN>
__device__ __forceinline__ void nv_quotients(float (&v)[kN], float T, float amax) {
  const float r = __frcp_rn(T);
  float y[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) y[i] = div_given_rcp(v[i], T, r);
  if (nv_plain<false>(T, amax)) {
#pragma unroll
    for (int i = 0; i < kN; i += 4) {
      const float4 q = div4(v[i], v[i + 1], v[i + 2], v[i + 3], T);
      y[i] = q.x, y[i + 1] = q.y, y[i + 2] = q.z, y[i + 3] = q.w;
    }
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = y[i];
}

// pairs of float32 in one 64-bit register: two roundings an instruction
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}

// Codes of eight values of a block under its NVFP4 scale T, e2m1(x / T), where !nv_plain; r is 1 / T
// correctly rounded.  Takes the values negated (nx = -x), as the packed residuals q T - x want them;
// the steps are div_given_rcp's.  For x of 8 bits (bf16) one step gives the same codes: it leaves
// q1 = fl(x / T (1 + e)), |e| < 2^-46, which can fall on another side of a code's border t (an odd
// multiple of 1/4 up to 5, t = J 2^n with J = 1, 3, 5, 7) than fl(x / T) only if x / T is that close to
// the middle M of t and a neighbour.  As integers, M = J 2^s +- 1 of 25 bits (s >= 22), T of 24, x of 8
// at the same scale: M T would be within 8 of a multiple of 2^41.  Modulo 2^22 that makes T = c 2^22 + d
// with |d| <= 8 and c = 2, 3 or 4; what remains is J d 2^s +- c 2^22 +- d within 8 of 0, so
// J d 2^(s - 22) = -+ c, which has one solution: J = 1, s = 24, c = 4, d = -1, T = 2^24 - 1 (a run over
// all T and M finds no other).
template <bool kBf16>
__device__ __forceinline__ uint32_t nv_codes8_common(const float (&nx)[8], float T, float r) {
  const uint64_t T2 = f32x2(T, T), nr2 = f32x2(-r, -r);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint64_t n2 = f32x2(nx[i], nx[i + 1]);
    uint64_t q = mul_f32x2(n2, nr2);
    if constexpr (!kBf16) q = fma_f32x2(fma_f32x2(q, T2, n2), nr2, q);
    q = fma_f32x2(fma_f32x2(q, T2, n2), nr2, q);
    asm("mov.b64 {%0, %1}, %2;" : "=f"(y[i]), "=f"(y[i + 1]) : "l"(q));
  }
  return e2m1x8_rn(y, 1.f);
}
// the same by plain division, zeros for T = 0
__device__ __forceinline__ uint32_t nv_codes8_plain(const float (&nx)[8], float T) {
  const float4 a = div4(nx[0], nx[1], nx[2], nx[3], -T), b = div4(nx[4], nx[5], nx[6], nx[7], -T);
  const float y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  return e2m1x8_rn(y, 1.f);
}

// 2^(byte - 127); byte 255 is NaN, byte 0 the subnormal 2^-127
__device__ __forceinline__ float ue8m0_value(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FC00000u) : (byte == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23));
}

// the values of kN packed codes (the even element in the low nibble); exact in f16
template <int kN>
__device__ __forceinline__ void e2m1_values(uint32_t word, float (&v)[kN]) {
#pragma unroll
  for (int i = 0; i < kN / 2; ++i) {
    uint32_t h;
    asm("{\n\t.reg .b8 q;\n\t"
        "cvt.u8.u32 q, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, q;\n\t}\n"
        : "=r"(h)
        : "r"(word >> (8 * i)));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// larger of two pairs of bf16, NaNs left out
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// largest magnitude of eight bf16, NaNs left out (0 if there is nothing else)
__device__ __forceinline__ float bf16x8_amax(const uint4& u) {
  const uint32_t a = bf16x2_max(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu), b = bf16x2_max(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu);
  const uint32_t m = bf16x2_max(a, b);
  return fmaxf(fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u)), 0.f);
}

// a pair of bf16 as floats, or as floats negated (a shift and add, as one instruction, flips the sign)
template <bool kNeg>
__device__ __forceinline__ void bf16x2_floats(uint32_t w, float& lo, float& hi) {
  lo = __uint_as_float((w << 16) + (kNeg ? 0x80000000u : 0u));
  hi = __uint_as_float((w & 0xFFFF0000u) ^ (kNeg ? 0x80000000u : 0u));
}

// eight values as they lie in memory (16 bytes of bf16, 32 of float32), and as floats
template <bool kBf16>
struct Raw8;
template <>
struct Raw8<true> {
  uint4 u;
  __device__ __forceinline__ void load(const void* x, int64_t at) {
    u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at));
  }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ float amax() const { return bf16x8_amax(u); }
  template <bool kNeg>  // (negated: as nv_codes8 takes them)
  __device__ __forceinline__ void values(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) bf16x2_floats<kNeg>(w[i], v[2 * i], v[2 * i + 1]);
  }
};
template <>
struct Raw8<false> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* x, int64_t at) {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
    a = __ldg(s);
    b = __ldg(s + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ float amax() const {
    const float m0 = fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w)));
    const float m1 = fmaxf(fmaxf(fabsf(b.x), fabsf(b.y)), fmaxf(fabsf(b.z), fabsf(b.w)));
    return fmaxf(fmaxf(m0, m1), 0.f);
  }
  template <bool kNeg>
  __device__ __forceinline__ void values(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    if constexpr (kNeg) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = -v[i];
    }
  }
};

__device__ __forceinline__ uint32_t fp4_bf16x2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

}  // namespace csa
