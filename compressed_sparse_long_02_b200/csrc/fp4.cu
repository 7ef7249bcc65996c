// fp4.cu -- microscaled 4-bit matrices: encoding and decoding in the layout the product
// (fp4_gemm.cu) streams, and the re-layout of row-major scales.
//
// Formats (include/csa.h, csa_fp4_format):
//   MXFP4: E2M1 codes, one UE8M0 scale per 32 elements -- the rule of mxfp4.cuh.
//   NVFP4: E2M1 codes, one E4M3 scale s per 16 elements and one float32 scale g per tensor:
//          s = e4m3(amax / (6 g)), T = s g, code = e2m1(x / T); every step one float32
//          rounding, so the bytes are a function of the input bits alone.
//
// Scales are stored as the tensor core reads them: blocks of 128 rows x 4 scales, 512 bytes,
// the scale (r, b) of a block at byte (r % 32) * 16 + (r / 32) * 4 + b; row blocks outermost.
// So one warp takes the four rows r, r + 32, r + 64, r + 96 of a row block over 256 columns:
// the four rows' scales of an atom are 16 consecutive bytes, and four loads are in flight per
// lane.  Rows and columns that pad a block get scale bytes of zero.
//
// All three kernels are bound by HBM: 2 or 4 bytes read and 17/32 or 9/16 written per element.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "fp4.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace csa {
namespace {

constexpr int kFp4Threads = 256;
constexpr int kChunk = 256;  // columns of a warp's task: 8 per lane

struct Fp4Shape {
  int64_t rows;
  int cols;
  int64_t ld;      // elements between rows of the unencoded matrix
  int n_atoms;     // scale atoms (4 scales) per row
  int n_chunks;    // ceil(padded columns / 256)
  int64_t n_tasks; // row blocks * 32 * n_chunks
};

template <bool kBf16, bool kNv>
__global__ void __launch_bounds__(kFp4Threads) fp4_quantize_kernel(const void* __restrict__ x, Fp4Shape p,
                                                                   const float* __restrict__ tensor_scale,
                                                                   uint8_t* __restrict__ packed,
                                                                   uint8_t* __restrict__ scales) {
  griddep_enter();
  const int lane = threadIdx.x & 31;
  const int64_t warp0 = (static_cast<int64_t>(blockIdx.x) * kFp4Threads + threadIdx.x) >> 5;
  const int64_t n_warps = static_cast<int64_t>(gridDim.x) * (kFp4Threads / 32);
  const float g = kNv ? __ldg(tensor_scale) : 1.f;
  const float six_g = 6.f * g;
  for (int64_t task = warp0; task < p.n_tasks; task += n_warps) {
    const int chunk = static_cast<int>(task % p.n_chunks);
    const int64_t rest = task / p.n_chunks;
    const int r32 = static_cast<int>(rest & 31);
    const int64_t rb = rest >> 5;
    const int col = chunk * kChunk + lane * 8;
    float v[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = rb * 128 + r32 + 32 * i;
      if (row < p.rows && col < p.cols) {  // cols is a multiple of 32: a lane's 8 are all in or all out
        fp4_load8<kBf16>(x, row * p.ld + col, v[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
      }
    }
    uint32_t sword[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = rb * 128 + r32 + 32 * i;
      const bool in = row < p.rows && col < p.cols;
      float am = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) am = fmaxf(am, fabsf(v[i][e]));
      am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
      uint32_t word, byte;
      if constexpr (kNv) {
        byte = nv_scale_byte(am, six_g);
        word = nv_codes8(v[i], e4m3_value(byte) * g);
      } else {
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
        const int E = mx_block_exponent(am);
        word = e2m1x8_rn(v[i], mx_pow2_neg(E));
        byte = static_cast<uint32_t>(E + 127);
      }
      if (in) reinterpret_cast<uint32_t*>(packed)[(row * p.cols + col) >> 3] = word;
      // the four scale bytes of an atom (16 lanes; NVFP4: 8) into one word, in every lane
      constexpr int kStep = kNv ? 2 : 4;  // lanes per block
      uint32_t w = in ? byte << (8 * ((lane / kStep) & 3)) : 0u;
      w |= __shfl_xor_sync(0xffffffffu, w, kStep);
      w |= __shfl_xor_sync(0xffffffffu, w, 2 * kStep);
      sword[i] = w;
    }
    constexpr int kLanes = kNv ? 8 : 16;  // lanes per atom
    const int atom = chunk * (32 / kLanes) + lane / kLanes;
    if (lane % kLanes == 0 && atom < p.n_atoms)
      *reinterpret_cast<uint4*>(scales + fp4_atom_offset(rb, atom, p.n_atoms) + r32 * 16) =
          make_uint4(sword[0], sword[1], sword[2], sword[3]);
  }
}

template <bool kBf16, bool kNv>
__global__ void __launch_bounds__(kFp4Threads) fp4_dequantize_kernel(const uint8_t* __restrict__ packed,
                                                                     const uint8_t* __restrict__ scales, Fp4Shape p,
                                                                     const float* __restrict__ tensor_scale,
                                                                     void* __restrict__ out) {
  griddep_enter();
  const int lane = threadIdx.x & 31;
  const int64_t warp0 = (static_cast<int64_t>(blockIdx.x) * kFp4Threads + threadIdx.x) >> 5;
  const int64_t n_warps = static_cast<int64_t>(gridDim.x) * (kFp4Threads / 32);
  const float g = kNv ? __ldg(tensor_scale) : 1.f;
  constexpr int kLanes = kNv ? 8 : 16;
  constexpr int kStep = kNv ? 2 : 4;
  for (int64_t task = warp0; task < p.n_tasks; task += n_warps) {
    const int chunk = static_cast<int>(task % p.n_chunks);
    const int64_t rest = task / p.n_chunks;
    const int r32 = static_cast<int>(rest & 31);
    const int64_t rb = rest >> 5;
    const int col = chunk * kChunk + lane * 8;
    if (rb * 128 + r32 >= p.rows || col >= p.cols) continue;  // no shuffles below: lanes may part
    const int atom = chunk * (32 / kLanes) + lane / kLanes;
    const uint4 sv = __ldg(reinterpret_cast<const uint4*>(scales + fp4_atom_offset(rb, atom, p.n_atoms) + r32 * 16));
    const uint32_t sw[4] = {sv.x, sv.y, sv.z, sv.w};
    uint32_t word[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = rb * 128 + r32 + 32 * i;
      word[i] = row < p.rows ? __ldg(reinterpret_cast<const uint32_t*>(packed) + ((row * p.cols + col) >> 3)) : 0u;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = rb * 128 + r32 + 32 * i;
      if (row >= p.rows) break;
      const uint32_t byte = (sw[i] >> (8 * ((lane / kStep) & 3))) & 0xFFu;
      const float T = kNv ? e4m3_value(byte) * g : ue8m0_value(byte);
      float v[8];
      e2m1x8_values(word[i], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= T;
      fp4_store8<kBf16>(out, row * p.ld + col, v);
    }
  }
}

// Row-major scale bytes [rows, nb] into the blocked layout: a thread writes the 4 bytes of one
// (row, atom), zeros where the row or the scale only pads a block.
__global__ void __launch_bounds__(kFp4Threads) fp4_pack_scales_kernel(const uint8_t* __restrict__ in, int64_t rows,
                                                                      int nb, int n_atoms, int64_t n_words,
                                                                      uint32_t* __restrict__ out) {
  griddep_enter();
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kFp4Threads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kFp4Threads + threadIdx.x; i < n_words; i += stride) {
    const int w = static_cast<int>(i & 127);
    const int64_t blk = i >> 7;
    const int atom = static_cast<int>(blk % n_atoms);
    const int64_t row = blk / n_atoms * 128 + (w & 3) * 32 + (w >> 2);
    uint32_t v = 0;
    if (row < rows) {
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (atom * 4 + b < nb) v |= static_cast<uint32_t>(in[row * nb + atom * 4 + b]) << (8 * b);
    }
    out[i] = v;
  }
}

Fp4Shape fp4_shape(bool nv, int64_t rows, int cols, int64_t ld) {
  Fp4Shape p{};
  p.rows = rows;
  p.cols = cols;
  p.ld = ld;
  p.n_atoms = fp4_atoms(nv, cols);
  p.n_chunks = (cols + kChunk - 1) / kChunk;
  p.n_tasks = (rows + 127) / 128 * 32 * p.n_chunks;
  return p;
}

// one warp per task up to eight CTAs per SM, a loop beyond
unsigned fp4_grid(int64_t n_tasks) {
  const int64_t blocks = (n_tasks + kFp4Threads / 32 - 1) / (kFp4Threads / 32);
  const int64_t cap = static_cast<int64_t>(num_sms()) * 8;
  return static_cast<unsigned>(blocks < cap ? blocks : cap);
}

}  // namespace

size_t fp4_scale_bytes(bool nv, int64_t rows, int cols) {
  return static_cast<size_t>((rows + 127) / 128) * fp4_atoms(nv, cols) * 512;
}

cudaError_t launch_fp4_quantize(bool nv, const void* x, int in_bf16, int64_t rows, int cols, int64_t ld,
                                const float* tensor_scale, uint8_t* packed, uint8_t* scales, cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  const Fp4Shape p = fp4_shape(nv, rows, cols, ld);
  const dim3 grid(fp4_grid(p.n_tasks)), block(kFp4Threads);
  auto k = nv ? (in_bf16 ? fp4_quantize_kernel<true, true> : fp4_quantize_kernel<false, true>)
              : (in_bf16 ? fp4_quantize_kernel<true, false> : fp4_quantize_kernel<false, false>);
  return launch_pdl(k, grid, block, 0, s, x, p, tensor_scale, packed, scales);
}

cudaError_t launch_fp4_dequantize(bool nv, const uint8_t* packed, const uint8_t* scales, const float* tensor_scale,
                                  int64_t rows, int cols, int out_bf16, void* out, int64_t ld, cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  const Fp4Shape p = fp4_shape(nv, rows, cols, ld);
  const dim3 grid(fp4_grid(p.n_tasks)), block(kFp4Threads);
  auto k = nv ? (out_bf16 ? fp4_dequantize_kernel<true, true> : fp4_dequantize_kernel<false, true>)
              : (out_bf16 ? fp4_dequantize_kernel<true, false> : fp4_dequantize_kernel<false, false>);
  return launch_pdl(k, grid, block, 0, s, packed, scales, p, tensor_scale, out);
}

cudaError_t launch_fp4_pack_scales(bool nv, const uint8_t* in, int64_t rows, int cols, uint8_t* out, cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  const int n_atoms = fp4_atoms(nv, cols);
  const int64_t n_words = (rows + 127) / 128 * n_atoms * 128;
  const int64_t blocks = (n_words + kFp4Threads - 1) / kFp4Threads;
  const int64_t cap = static_cast<int64_t>(num_sms()) * 8;
  return launch_pdl(fp4_pack_scales_kernel, dim3(static_cast<unsigned>(blocks < cap ? blocks : cap)), dim3(kFp4Threads),
                    0, s, in, rows, cols / fp4_block(nv), n_atoms, n_words, reinterpret_cast<uint32_t*>(out));
}

}  // namespace csa
