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

// NVFP4 scale byte of a block: e4m3(amax / (6 g)), to nearest even, at most 448
__device__ __forceinline__ uint32_t nv_scale_byte(float amax, float six_g) {
  return __nv_cvt_float_to_fp8(__fdiv_rn(amax, six_g), __NV_SATFINITE, __NV_E4M3);
}

// Codes of eight values under the NVFP4 scale T: e2m1(x / T), zeros if T is zero
__device__ __forceinline__ uint32_t nv_codes8(const float (&v)[8], float T) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = T > 0.f ? __fdiv_rn(v[i], T) : 0.f;
  return e2m1x8_rn(y, 1.f);
}

// 2^(byte - 127); byte 255 is NaN, byte 0 the subnormal 2^-127
__device__ __forceinline__ float ue8m0_value(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FC00000u) : (byte == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23));
}

// the values of eight packed codes (the even element in the low nibble); exact in f16
__device__ __forceinline__ void e2m1x8_values(uint32_t word, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
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

template <bool kBf16>
__device__ __forceinline__ void fp4_load8(const void* x, int64_t at, float (&v)[8]) {
  if constexpr (kBf16) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
    const float4 a = __ldg(s), b = __ldg(s + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

__device__ __forceinline__ uint32_t fp4_bf16x2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// larger of two pairs of bf16, NaNs left out
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

template <bool kBf16>
__device__ __forceinline__ void fp4_store8(void* out, int64_t at, const float (&v)[8]) {
  if constexpr (kBf16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) =
        make_uint4(fp4_bf16x2(v[0], v[1]), fp4_bf16x2(v[2], v[3]), fp4_bf16x2(v[4], v[5]), fp4_bf16x2(v[6], v[7]));
  } else {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
    d[0] = make_float4(v[0], v[1], v[2], v[3]);
    d[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

}  // namespace csa
