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
// So one warp takes the four rows r, r + 32, r + 64, r + 96 of a row block over its columns:
// the four rows' scales of an atom are 16 consecutive bytes, and the loads of all four are in
// flight before the first is used.  Rows and columns that pad a block get scale bytes of zero.
//
// All three kernels are bound by HBM: 2 or 4 bytes read and 17/32 or 9/16 written per element.
// 8192 x 32768 bf16 on one B200: MXFP4 encoding 100 us (6.8 TB/s, the copy rate) and decoding 105;
// NVFP4 112 us (6.2 TB/s: about 180 instructions for 16 values of a lane, MXFP4 160) and 106.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>
#include <utility>

#include "fp4.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace csa {
namespace {

constexpr int kFp4Threads = 256;

struct Fp4Shape {
  int64_t rows;
  int cols;
  int64_t ld;      // elements between rows of the unencoded matrix
  int n_atoms;     // scale atoms (4 scales) per row
  int n_chunks;    // columns in units of a warp's task
  int64_t n_rows32; // row blocks * 32
};

// A warp's tasks: (row, chunk) pairs, chunks fastest, `n_warps` apart -- stepped without a division
struct Task {
  int64_t row, step_row;
  int chunk, step_chunk;
  __device__ Task(int64_t warp, int64_t n_warps, int n_chunks)
      : row(warp / n_chunks), step_row(n_warps / n_chunks), chunk(static_cast<int>(warp % n_chunks)),
        step_chunk(static_cast<int>(n_warps % n_chunks)) {}
  __device__ void next(int n_chunks) {
    row += step_row;
    chunk += step_chunk;
    if (chunk >= n_chunks) {
      chunk -= n_chunks;
      ++row;
    }
  }
};

// What a lane encodes of one row: 32 bytes, 16 bf16 or 8 float32 (half or a quarter of an MXFP4
// block, a whole NVFP4 block or half of one).
template <bool kBf16>
constexpr int kEncodePer = kBf16 ? 16 : 8;
template <bool kBf16>
constexpr int kEncodeChunk = 32 * kEncodePer<kBf16>;  // columns of a warp's task

template <bool kBf16, bool kNv>
struct RowTask {
  static constexpr int kPer = kEncodePer<kBf16>, kUnits = kPer / 8, kBlk = kNv ? 16 : 32;
  static constexpr int kBlkLanes = kBlk / kPer, kAtomLanes = 4 * kBlkLanes;
  Raw8<kBf16> raw[kUnits];

  __device__ __forceinline__ void load(const void* x, int64_t at, bool in) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      if (in)
        raw[u].load(x, at + 8 * u);
      else
        raw[u].zero();
    }
  }
  // stores the codes (where `in`) and returns the atom's four scale bytes, in each of its lanes;
  // `plain` is set where the codes need plain division: see encode_plain
  __device__ __forceinline__ uint32_t encode(const NvScale& nv, uint8_t* packed, int64_t at, bool in, bool& plain) const {
    const int lane = threadIdx.x & 31;
    float am = raw[0].amax();
#pragma unroll
    for (int u = 1; u < kUnits; ++u) am = fmaxf(am, raw[u].amax());
#pragma unroll
    for (int o = 1; o < kBlkLanes; o <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
    uint32_t byte, word[kUnits];
    float T = 0.f;
    if constexpr (kNv) {
      byte = nv.byte(am);
      T = e4m3_value(byte) * nv.g;
      plain = T != 0.f && nv_plain<kBf16>(T, am);
    } else {
      const int E = mx_block_exponent(am);
      T = mx_pow2_neg(E);
      byte = static_cast<uint32_t>(E + 127);
    }
    const float r = kNv ? __frcp_rn(T) : 0.f;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      float v[8];
      raw[u].template values<kNv>(v);
      word[u] = kNv ? (T == 0.f ? 0u : nv_codes8_common<kBf16>(v, T, r)) : e2m1x8_rn(v, T);
    }
    if (in) {
      if constexpr (kUnits == 2)
        *reinterpret_cast<uint2*>(packed + at / 2) = make_uint2(word[0], word[1]);
      else
        *reinterpret_cast<uint32_t*>(packed + at / 2) = word[0];
    }
    uint32_t w = in ? byte << (8 * ((lane / kBlkLanes) & 3)) : 0u;
    w |= __shfl_xor_sync(0xffffffffu, w, kBlkLanes);
    w |= __shfl_xor_sync(0xffffffffu, w, 2 * kBlkLanes);
    return w;
  }
};

// The codes of a lane's share of a row by plain division, over what encode() stored (out of line, from
// memory again: extreme scales only, and the common path keeps no values for it).
template <bool kBf16>
static __device__ __noinline__ void encode_plain(const void* x, int64_t at, float T, uint8_t* packed, int64_t at_codes) {
#pragma unroll 1
  for (int u = 0; u < kEncodePer<kBf16>; u += 8) {
    Raw8<kBf16> raw;
    raw.load(x, at + u);
    float v[8];
    raw.template values<true>(v);
    *reinterpret_cast<uint32_t*>(packed + (at_codes + u) / 2) = nv_codes8_plain(v, T);
  }
}

// (four CTAs an SM asked for where it pays: NVFP4 from float32, 8192 x 32768, 198 -> 186 us; the other
// three reach four by themselves, 0 being no request)
template <bool kBf16, bool kNv>
__global__ void __launch_bounds__(kFp4Threads, kNv && !kBf16 ? 4 : 0) fp4_quantize_kernel(const void* __restrict__ x, Fp4Shape p,
                                                                   const float* __restrict__ tensor_scale,
                                                                   uint8_t* __restrict__ packed,
                                                                   uint8_t* __restrict__ scales) {
  using RT = RowTask<kBf16, kNv>;
  griddep_enter();
  const int lane = threadIdx.x & 31;
  const int64_t warp0 = (static_cast<int64_t>(blockIdx.x) * kFp4Threads + threadIdx.x) >> 5;
  const int64_t n_warps = static_cast<int64_t>(gridDim.x) * (kFp4Threads / 32);
  const NvScale nv(kNv ? __ldg(tensor_scale) : 1.f);
  for (Task t(warp0, n_warps, p.n_chunks); t.row < p.n_rows32; t.next(p.n_chunks)) {
    const int r32 = t.row & 31;
    const int64_t row0 = (t.row >> 5) * 128 + r32;
    const int col = t.chunk * kEncodeChunk<kBf16> + lane * RT::kPer;
    const bool in = col < p.cols;  // cols is a multiple of 32: a lane's columns are all in or all out
    uint32_t w[4] = {0, 0, 0, 0};
    bool plain[4] = {false, false, false, false};
    if (row0 + 96 < p.rows) {
      RT rt[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) rt[i].load(x, (row0 + 32 * i) * p.ld + col, in);  // every load first
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = rt[i].encode(nv, packed, (row0 + 32 * i) * p.cols + col, in, plain[i]);
    } else {  // the last row block: one row at a time, so that rows that only pad it cost nothing
      RT rt;
      rt.load(x, row0 * p.ld + col, in && row0 < p.rows);
#pragma unroll 1
      for (int64_t row = row0; row < p.rows; row += 32) {
        RT next;
        next.load(x, (row + 32) * p.ld + col, in && row + 32 < p.rows);
        bool pl = false;
        const uint32_t v = rt.encode(nv, packed, row * p.cols + col, in, pl);
        rt = next;
        const int i = static_cast<int>((row - row0) / 32);
        plain[0] |= i == 0 && pl, plain[1] |= i == 1 && pl, plain[2] |= i == 2 && pl;
        w[0] = i == 0 ? v : w[0];
        w[1] = i == 1 ? v : w[1];
        w[2] = i == 2 ? v : w[2];
      }
    }
    const int atom = (t.chunk * 32 + lane) / RT::kAtomLanes;
    if (lane % RT::kAtomLanes == 0 && atom < p.n_atoms)
      *reinterpret_cast<uint4*>(scales + fp4_atom_offset(t.row >> 5, atom, p.n_atoms) + r32 * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (kNv) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t row = row0 + 32 * i;
        const uint32_t byte = (w[i] >> (8 * ((lane / RT::kBlkLanes) & 3))) & 0xFFu;
        if (plain[i] && in) encode_plain<kBf16>(x, row * p.ld + col, e4m3_value(byte) * nv.g, packed, row * p.cols + col);
      }
    }
  }
}

// Decoding writes 2 or 4 bytes for every half byte read, so the mapping follows the stores: a lane
// takes 16 bytes of output at a time (8 bf16 or 4 float32), twice per row, each warp store
// contiguous.
template <bool kBf16>
constexpr int kDecodeChunk = kBf16 ? 512 : 256;  // columns of a warp's task

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
  constexpr int kPer = kBf16 ? 8 : 4, kBlk = kNv ? 16 : 32;
  using Codes = typename std::conditional<kBf16, uint32_t, uint16_t>::type;
  for (Task t(warp0, n_warps, p.n_chunks); t.row < p.n_rows32; t.next(p.n_chunks)) {
    const int r32 = t.row & 31;
    const int64_t rb = t.row >> 5;
    if (rb * 128 + r32 >= p.rows) continue;
    uint4 sv[2];
    Codes word[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // every load first
      const int col = t.chunk * kDecodeChunk<kBf16> + (h * 32 + lane) * kPer;
      if (col < p.cols)
        sv[h] = __ldg(reinterpret_cast<const uint4*>(scales + fp4_atom_offset(rb, col / (4 * kBlk), p.n_atoms) + r32 * 16));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t row = rb * 128 + r32 + 32 * i;
        word[h][i] = row < p.rows && col < p.cols
                         ? __ldg(reinterpret_cast<const Codes*>(packed) + (row * p.cols + col) / kPer)
                         : static_cast<Codes>(0);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int col = t.chunk * kDecodeChunk<kBf16> + (h * 32 + lane) * kPer;
      if (col >= p.cols) continue;
      const uint32_t sw[4] = {sv[h].x, sv[h].y, sv[h].z, sv[h].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t row = rb * 128 + r32 + 32 * i;
        if (row >= p.rows) break;
        const uint32_t byte = (sw[i] >> (8 * (col / kBlk & 3))) & 0xFFu;
        const float T = kNv ? e4m3_value(byte) * g : ue8m0_value(byte);
        float v[kPer];
        e2m1_values<kPer>(word[h][i], v);
#pragma unroll
        for (int e = 0; e < kPer; ++e) v[e] *= T;
        if constexpr (kBf16)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + row * p.ld + col) =
              make_uint4(fp4_bf16x2(v[0], v[1]), fp4_bf16x2(v[2], v[3]), fp4_bf16x2(v[4], v[5]), fp4_bf16x2(v[6], v[7]));
        else
          *reinterpret_cast<float4*>(static_cast<float*>(out) + row * p.ld + col) = make_float4(v[0], v[1], v[2], v[3]);
      }
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

Fp4Shape fp4_shape(bool nv, int64_t rows, int cols, int64_t ld, int chunk) {
  Fp4Shape p{};
  p.rows = rows;
  p.cols = cols;
  p.ld = ld;
  p.n_atoms = fp4_atoms(nv, cols);
  p.n_chunks = (cols + chunk - 1) / chunk;
  p.n_rows32 = (rows + 127) / 128 * 32;
  return p;
}

// One warp per task up to `per_sm` CTAs per SM (four run at once), a loop beyond.  Measured on 8192 x
// 32768 (us; 8 / 16 / 64 per SM): MXFP4 from float32 183 / 182 / 172, from bf16 102 / 101 / 99.5; NVFP4,
// whose warps have more to set up, 187 / 186 / 192 and 113 / 112 / 113; decoding to bf16 119 / 114 / 105.
unsigned fp4_grid(int64_t n_tasks, int per_sm) {
  const int64_t blocks = (n_tasks + kFp4Threads / 32 - 1) / (kFp4Threads / 32);
  return static_cast<unsigned>(std::min<int64_t>(blocks, static_cast<int64_t>(num_sms()) * per_sm));
}

// A grid that fills the GPU asks for SMs that give all of their memory to L1: an SM's loads in flight,
// 4 KB a warp, need room there, and a grid that starts early, behind one that used the whole shared
// memory, keeps that one's split otherwise (the grouped projection of 8192 tokens: 345 us, 307 with the
// request).  A smaller one has few loads in flight and would only wait for the change (the projection
// of 32 tokens: 19.2 us, 21.1 with the request).
template <typename... KArgs, typename... Args>
cudaError_t launch_rows(void (*k)(KArgs...), unsigned grid, cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kFp4Threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributePreferredSharedMemoryCarveout;
  attr[1].val.sharedMemCarveout = cudaSharedmemCarveoutMaxL1;
  cfg.attrs = attr;
  cfg.numAttrs = grid >= static_cast<unsigned>(num_sms()) * 8 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, std::forward<Args>(args)...);
}

}  // namespace

size_t fp4_scale_bytes(bool nv, int64_t rows, int cols) {
  return static_cast<size_t>((rows + 127) / 128) * fp4_atoms(nv, cols) * 512;
}

cudaError_t launch_fp4_quantize(bool nv, const void* x, int in_bf16, int64_t rows, int cols, int64_t ld,
                                const float* tensor_scale, uint8_t* packed, uint8_t* scales, cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  const Fp4Shape p = fp4_shape(nv, rows, cols, ld, in_bf16 ? kEncodeChunk<true> : kEncodeChunk<false>);
  const unsigned grid = fp4_grid(p.n_rows32 * p.n_chunks, nv ? 16 : 64);
  auto k = nv ? (in_bf16 ? fp4_quantize_kernel<true, true> : fp4_quantize_kernel<false, true>)
              : (in_bf16 ? fp4_quantize_kernel<true, false> : fp4_quantize_kernel<false, false>);
  return launch_rows(k, grid, s, x, p, tensor_scale, packed, scales);
}

cudaError_t launch_fp4_dequantize(bool nv, const uint8_t* packed, const uint8_t* scales, const float* tensor_scale,
                                  int64_t rows, int cols, int out_bf16, void* out, int64_t ld, cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  const Fp4Shape p = fp4_shape(nv, rows, cols, ld, out_bf16 ? kDecodeChunk<true> : kDecodeChunk<false>);
  const unsigned grid = fp4_grid(p.n_rows32 * p.n_chunks, 64);
  auto k = nv ? (out_bf16 ? fp4_dequantize_kernel<true, true> : fp4_dequantize_kernel<false, true>)
              : (out_bf16 ? fp4_dequantize_kernel<true, false> : fp4_dequantize_kernel<false, false>);
  return launch_rows(k, grid, s, packed, scales, p, tensor_scale, out);
}

cudaError_t launch_fp4_pack_scales(bool nv, const uint8_t* in, int64_t rows, int cols, uint8_t* out, cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  const int n_atoms = fp4_atoms(nv, cols);
  const int64_t n_words = (rows + 127) / 128 * n_atoms * 128;
  const unsigned grid = fp4_grid((n_words + 31) / 32, 8);
  return launch_pdl(fp4_pack_scales_kernel, dim3(grid), dim3(kFp4Threads), 0, s, in, rows,
                    cols / fp4_block(nv), n_atoms, n_words, reinterpret_cast<uint32_t*>(out));
}

}  // namespace csa
