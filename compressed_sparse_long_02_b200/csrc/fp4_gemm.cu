// fp4_gemm.cu -- product of two microscaled 4-bit matrices on the block-scaled tensor cores.
//
//   y[m, g N + n] = gx gw sum_k X[m, g K + k] W[g N + n, k]      (g < G groups)
//
// X [M, G K] and W [G N, K] hold E2M1 codes with a scale per 32 (MXFP4) or 16 (NVFP4)
// elements, in the layout of fp4.cu; gx, gw are the float32 tensor scales (NVFP4).  The
// tensor core multiplies the codes and applies both scales per K = 64 step
// (tcgen05.mma kind::mxf4 / kind::mxf4nvf4, block_scale), accumulating in float32 in TMEM.
//
// The weights go on the MMA's M axis (128 output features a tile) and the tokens on its N
// axis (kBN a tile), so one kernel serves a single decode token (kBN = 32: the weights are
// streamed once, nothing is padded to 128 rows) and a prefill (kBN = 256).  A K slab is 256
// elements = 128 bytes a row, one swizzle row.
//
// Roles (320 threads): warp 0 issues the loads (codes by TMA boxes, scale atoms by bulk
// copies), warp 1 owns TMEM and one thread of it copies the slab's scales to TMEM and issues
// the MMAs, warps 2-9 write the results (two warps per TMEM lane quarter, half of the tile's
// tokens each; a lane holds one output feature, so a warp's store covers 32 consecutive
// features of a token).
//
// With few tiles the K axis is split over the S CTAs of a cluster: each accumulates its
// share, puts the float32 partial tile into its shared memory, and CTA r adds the S partials
// of its tokens in rank order (the sum does not depend on timing).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "fp4.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "tmap.h"

namespace csa {
namespace {

constexpr int kTileN = 128;          // output features of a tile (MMA M)
constexpr int kSlabBytes = 128;      // bytes of a row in a K slab: 256 elements
constexpr int kSlab = 2 * kSlabBytes;
constexpr int kThreads = 320;
constexpr int kEpiThreads = 256;
constexpr int kSfSlots = 4;          // TMEM slots of scale factors

template <bool kNv, int kBN>
struct Shape {
  static constexpr int kAtoms = kNv ? 4 : 2;                   // scale atoms of a slab per 128 rows
  static constexpr int kRowBlocks = kBN > 128 ? 2 : 1;         // 128-row scale blocks of the tokens
  static constexpr uint32_t kBytesW = kTileN * kSlabBytes;     // 16 KB
  static constexpr uint32_t kBytesX = kBN * kSlabBytes;
  static constexpr uint32_t kBytesSf = 512 * kAtoms * (1 + kRowBlocks);
  static constexpr uint32_t kStage = kBytesW + kBytesX + kBytesSf;
  static constexpr int kStages = static_cast<int>((224u * 1024u) / kStage) < 8 ? static_cast<int>((224u * 1024u) / kStage) : 8;
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStage + 512;
  static constexpr int kAcc = kBN > 128 ? 1 : 2;               // accumulators of kBN columns
  static constexpr uint32_t kSfCols = 4 * kAtoms * (1 + kRowBlocks);  // TMEM columns of a slab's scales
  static constexpr uint32_t kColSf = kAcc * kBN;
  static_assert(kColSf + kSfSlots * kSfCols <= 512, "TMEM budget");
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(kBN * kTileN * 4 <= kStages * kStage, "a partial tile fits in the ring");
};

struct LinearParams {
  int M, N, K, G;
  int n_blocks, m_blocks, tiles, splits;
  int x_atoms, w_atoms;   // scale atoms per row block of X and W
  int x_group_atoms;      // atoms of one group's K columns of X
  const uint8_t* x_scale;
  const uint8_t* w_scale;
  const float* gx;
  const float* gw;
  void* y;
  int64_t ldy;
  int vec4;               // rows of y allow 4-feature stores
  int32_t* err;
};

template <bool kBf16>
__device__ __forceinline__ void store_y(void* y, int64_t at, float v) {
  if constexpr (kBf16)
    static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(y)[at] = v;
}

template <bool kNv, int kBN, bool kBf16>
__global__ void __launch_bounds__(kThreads, 1)
    fp4_linear_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                      const LinearParams p) {
  using S = Shape<kNv, kBN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sW = smem;
  uint8_t* sX = sW + S::kStages * S::kBytesW;
  uint8_t* sSf = sX + S::kStages * S::kBytesX;
  uint64_t* full = reinterpret_cast<uint64_t*>(sSf + S::kStages * S::kBytesSf);
  uint64_t* empty = full + S::kStages;
  uint64_t* acc_full = empty + S::kStages;
  uint64_t* acc_empty = acc_full + S::kAcc;
  uint64_t* fin = acc_empty + S::kAcc;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(fin + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < S::kAcc; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 8);
    }
    mbar_init(fin, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_x);
    prefetch_tmap(&tm_w);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_enter();

  const int rank = static_cast<int>(blockIdx.x) % p.splits;
  const int first = static_cast<int>(blockIdx.x) / p.splits, step = static_cast<int>(gridDim.x) / p.splits;
  const int slabs = (p.K + kSlab - 1) / kSlab;
  const int slab0 = static_cast<int>(static_cast<int64_t>(slabs) * rank / p.splits);
  const int slab1 = static_cast<int>(static_cast<int64_t>(slabs) * (rank + 1) / p.splits);

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    if (lane == 0) {
      int j = 0;
      bool ok = true;
      for (int t = first; ok && t < p.tiles; t += step) {
        const int nb = t % p.n_blocks, mg = t / p.n_blocks;
        const int g = mg % p.G, m0 = (mg / p.G) * kBN;
        const int w_row = g * p.N + nb * kTileN;
        const int rb_x = m0 / 128;
        const int rbs = min(S::kRowBlocks, (p.M + 127) / 128 - rb_x);  // a ragged last tile may have one row block less
        const uint8_t* wsc = p.w_scale + fp4_atom_offset(w_row / 128, 0, p.w_atoms);
        const uint8_t* xsc = p.x_scale + fp4_atom_offset(rb_x, g * p.x_group_atoms, p.x_atoms);
        for (int sl = slab0; sl < slab1; ++sl, ++j) {
          const int st = j % S::kStages;
          if (!mbar_wait(&empty[st], ((j / S::kStages) & 1) ^ 1, p.err, abort_flag)) {
            ok = false;
            break;
          }
          const int atom0 = sl * S::kAtoms;
          const uint32_t sf_bytes = 512u * min(S::kAtoms, p.w_atoms - atom0);
          mbar_arrive_expect_tx(&full[st], S::kBytesW + S::kBytesX + sf_bytes * (1 + rbs));
          tma_load_2d(smem_u32(sW + st * S::kBytesW), &tm_w, &full[st], sl * kSlabBytes, w_row);
          tma_load_2d(smem_u32(sX + st * S::kBytesX), &tm_x, &full[st], g * (p.K / 2) + sl * kSlabBytes, m0);
          const uint32_t dst = smem_u32(sSf + st * S::kBytesSf);
          bulk_load(dst, wsc + atom0 * 512, sf_bytes, &full[st]);
          for (int rb = 0; rb < rbs; ++rb)
            bulk_load(dst + 512 * S::kAtoms * (1 + rb), xsc + fp4_atom_offset(rb, atom0, p.x_atoms), sf_bytes, &full[st]);
        }
      }
      // the last loads issued must have landed before this CTA's shared memory is reused or freed
      volatile int never = 0;
      for (int i = std::max(0, j - S::kStages); i < j; ++i)
        mbar_wait(&full[i % S::kStages], (i / S::kStages) & 1, p.err, &never);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      int j = 0, it = 0;
      bool ok = true;
      for (int t = first; ok && t < p.tiles; t += step, ++it) {
        const int buf = it % S::kAcc;
        if (!mbar_wait(&acc_empty[buf], ((it / S::kAcc) & 1) ^ 1, p.err, abort_flag)) break;
        tc_fence_after();
        const uint32_t acc = tmem + kBN * buf;
        for (int sl = slab0; sl < slab1; ++sl, ++j) {
          const int st = j % S::kStages;
          if (!mbar_wait(&full[st], (j / S::kStages) & 1, p.err, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int left = p.K - sl * kSlab;
          const int n_mma = min(4, (left + 63) / 64);
          const int atoms = min(S::kAtoms, p.w_atoms - sl * S::kAtoms);
          // scales: W in columns [0, 4 kAtoms) of the slot (4 per atom), then X (4 per atom and row block)
          const uint32_t sfw = tmem + S::kColSf + (j % kSfSlots) * S::kSfCols;
          const uint32_t sfx = sfw + 4 * S::kAtoms;
          const uint32_t src = smem_u32(sSf + st * S::kBytesSf);
          for (int a = 0; a < atoms; ++a) {
            tc_cp_32x128b_warpx4(sfw + 4 * a, smem_desc(src + 512 * a, 0, 128, kSwizzleNone));
            for (int rb = 0; rb < S::kRowBlocks; ++rb)
              tc_cp_32x128b_warpx4(sfx + 4 * (S::kRowBlocks * a + rb),
                                   smem_desc(src + 512 * (S::kAtoms * (1 + rb) + a), 0, 128, kSwizzleNone));
          }
          const uint32_t a0 = smem_u32(sW + st * S::kBytesW), b0 = smem_u32(sX + st * S::kBytesX);
          for (int kk = 0; kk < n_mma; ++kk) {
            const uint64_t da = smem_desc(a0 + 32 * kk, 16, 1024, kSwizzle128B);
            const uint64_t db = smem_desc(b0 + 32 * kk, 16, 1024, kSwizzle128B);
            const uint32_t accumulate = (sl > slab0 || kk > 0) ? 1u : 0u;
            if constexpr (kNv) {
              mma_nvf4(acc, da, db, idesc_nvf4(kTileN, kBN), accumulate, sfw + 4 * kk, sfx + 4 * S::kRowBlocks * kk);
            } else {
              const uint32_t id = 2 * (kk & 1);  // the byte of the scale column of this K = 64 step
              mma_mxf4(acc, da, db, idesc_mxf4(kTileN, kBN, id, id), accumulate, (sfw + 4 * (kk >> 1)) | (id << 30),
                       (sfx + 4 * S::kRowBlocks * (kk >> 1)) | (id << 30));
            }
          }
          tc_commit(&empty[st]);
        }
        if (ok) tc_commit(&acc_full[buf]);
      }
      tc_commit(fin);
      volatile int never = 0;
      mbar_wait(fin, 0, p.err, &never);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- results (warps 2-9)
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lane_base = static_cast<uint32_t>(32 * quarter) << 16;
    const float alpha = (p.gx ? __ldg(p.gx) : 1.f) * (p.gw ? __ldg(p.gw) : 1.f);
    float* part = reinterpret_cast<float*>(smem);  // [kBN tokens][128 features], split K only
    int it = 0;
    for (int t = first; t < p.tiles; t += step, ++it) {
      const int buf = it % S::kAcc;
      if (!warp_wait_sleep(&acc_full[buf], (it / S::kAcc) & 1, p.err, abort_flag)) break;
      tc_fence_after();
      const int nb = t % p.n_blocks, mg = t / p.n_blocks;
      const int g = mg % p.G, m0 = (mg / p.G) * kBN;
      const int f = 32 * quarter + lane, n = nb * kTileN + f;
      const int m_left = p.M - m0;
#pragma unroll 1
      for (int c = half * (kBN / 2); c < (half + 1) * (kBN / 2); c += 16) {
        if (c >= m_left) break;
        uint32_t v[16];
        tmem_ld16(tmem + lane_base + kBN * buf + c, v);
        tmem_wait_ld();
        if (p.splits > 1) {
#pragma unroll
          for (int i = 0; i < 16; ++i) part[(c + i) * kTileN + f] = __uint_as_float(v[i]);
        } else if (n < p.N) {
          const int64_t at = static_cast<int64_t>(m0 + c) * p.ldy + static_cast<int64_t>(g) * p.N + n;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c + i < m_left) store_y<kBf16>(p.y, at + i * p.ldy, __uint_as_float(v[i]) * alpha);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[buf]);
    }
  }

  if (p.splits > 1) {  // one tile per cluster: every CTA's partial, added in rank order
    cluster_sync_all();
    const int t = first;
    const int nb = t % p.n_blocks, mg = t / p.n_blocks;
    const int g = mg % p.G, m0 = (mg / p.G) * kBN;
    const int m_valid = min(kBN, p.M - m0);
    const int tok0 = m_valid * rank / p.splits, tok1 = m_valid * (rank + 1) / p.splits;
    const float alpha = (p.gx ? __ldg(p.gx) : 1.f) * (p.gw ? __ldg(p.gw) : 1.f);
    for (int i = threadIdx.x; i < (tok1 - tok0) * (kTileN / 4); i += kThreads) {
      const int tok = tok0 + i / (kTileN / 4), f = i % (kTileN / 4) * 4, n = nb * kTileN + f;
      const uint8_t* src = smem + (tok * kTileN + f) * 4;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int r = 0; r < p.splits; ++r) {
        const uint4 u = dsmem_ld4(dsmem_map(src, r));
        sum.x += __uint_as_float(u.x);
        sum.y += __uint_as_float(u.y);
        sum.z += __uint_as_float(u.z);
        sum.w += __uint_as_float(u.w);
      }
      const float o[4] = {sum.x * alpha, sum.y * alpha, sum.z * alpha, sum.w * alpha};
      const int64_t at = static_cast<int64_t>(m0 + tok) * p.ldy + static_cast<int64_t>(g) * p.N + n;
      if (p.vec4 && n + 3 < p.N) {
        if constexpr (kBf16)
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + at) = make_uint2(fp4_bf16x2(o[0], o[1]), fp4_bf16x2(o[2], o[3]));
        else
          *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) = make_float4(o[0], o[1], o[2], o[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < p.N) store_y<kBf16>(p.y, at + e, o[e]);
      }
    }
    cluster_sync_all();  // no CTA leaves while another still reads its partial
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <bool kNv, int kBN, bool kBf16>
cudaError_t launch_tile(const Fp4LinearArgs& a, LinearParams& p, cudaStream_t s) {
  using Sh = Shape<kNv, kBN>;
  static int smem_set[64];
  CUtensorMap tm_x, tm_w;
  const int64_t xb = static_cast<int64_t>(a.G) * a.K / 2, wb = a.K / 2;
  if (!encode_2d_u8(&tm_x, a.x_packed, xb, a.M, kSlabBytes, kBN, CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
  if (!encode_2d_u8(&tm_w, a.w_packed, wb, static_cast<uint64_t>(a.G) * a.N, kSlabBytes, kTileN, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  p.m_blocks = (a.M + kBN - 1) / kBN;
  const int64_t tiles = static_cast<int64_t>(p.m_blocks) * p.n_blocks * a.G;
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
  p.tiles = static_cast<int>(tiles);
  // Split K over 2, 4 or 8 CTAs while the tiles leave SMs idle and every CTA keeps two slabs or more.
  const int slabs = (a.K + kSlab - 1) / kSlab, sms = num_sms();
  p.splits = 1;
  while (p.splits < 8 && tiles * p.splits * 2 <= sms && slabs >= 4 * p.splits) p.splits *= 2;
  const int64_t clusters = p.splits > 1 ? tiles : std::min<int64_t>(tiles, sms);
  auto k = fp4_linear_kernel<kNv, kBN, kBf16>;
  const cudaError_t e = set_dyn_smem(reinterpret_cast<const void*>(k), Sh::kSmem, smem_set);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(clusters * p.splits)), block(kThreads);
  if (p.splits == 1) return launch_pdl(k, grid, block, Sh::kSmem, s, tm_x, tm_w, p);
  return launch_pdl_cluster(k, grid, block, Sh::kSmem, p.splits, s, tm_x, tm_w, p);
}

template <bool kNv, bool kBf16>
cudaError_t launch_shape(const Fp4LinearArgs& a, LinearParams& p, cudaStream_t s) {
  // tokens per tile: the smallest that takes them all, 256 beyond
  if (a.M <= 32) return launch_tile<kNv, 32, kBf16>(a, p, s);
  if (a.M <= 64) return launch_tile<kNv, 64, kBf16>(a, p, s);
  if (a.M <= 128) return launch_tile<kNv, 128, kBf16>(a, p, s);
  return launch_tile<kNv, 256, kBf16>(a, p, s);
}

}  // namespace

cudaError_t launch_fp4_linear(const Fp4LinearArgs& a, cudaStream_t s) {
  if (a.M == 0 || a.N == 0) return cudaSuccess;
  LinearParams p{};
  p.M = a.M;
  p.N = a.N;
  p.K = a.K;
  p.G = a.G;
  p.n_blocks = (a.N + kTileN - 1) / kTileN;
  p.x_atoms = fp4_atoms(a.nv, a.G * a.K);
  p.w_atoms = fp4_atoms(a.nv, a.K);
  p.x_group_atoms = a.G > 1 ? p.w_atoms : 0;
  p.x_scale = a.x_scale;
  p.w_scale = a.w_scale;
  p.gx = a.gx;
  p.gw = a.gw;
  p.y = a.y;
  p.ldy = a.ldy;
  p.vec4 = a.N % 4 == 0 && a.ldy % 4 == 0;
  p.err = device_error_word();
  if (p.err == nullptr) return cudaErrorUnknown;
  if (a.nv) return a.out_bf16 ? launch_shape<true, true>(a, p, s) : launch_shape<true, false>(a, p, s);
  return a.out_bf16 ? launch_shape<false, true>(a, p, s) : launch_shape<false, false>(a, p, s);
}

// ------------------------------------------------------------------ grouped output projection
// Scratch of the projection, 256-byte aligned pieces: o's codes and scales, z (bf16), z's
// codes and scales.
namespace {
struct ProjScratch {
  size_t o_packed, o_scale, z, z_packed, z_scale, bytes;
};
ProjScratch proj_scratch(bool nv, int T, int64_t HD, int64_t GR) {
  ProjScratch w{};
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t r = at;
    at += (n + 255) / 256 * 256;
    return r;
  };
  w.o_packed = take(static_cast<size_t>(T) * HD / 2);
  w.o_scale = take(fp4_scale_bytes(nv, T, static_cast<int>(HD)));
  w.z = take(static_cast<size_t>(T) * GR * 2);
  w.z_packed = take(static_cast<size_t>(T) * GR / 2);
  w.z_scale = take(fp4_scale_bytes(nv, T, static_cast<int>(GR)));
  w.bytes = at;
  return w;
}
}  // namespace

size_t fp4_proj_workspace_bytes(bool nv, int T, int64_t HD, int64_t GR) { return proj_scratch(nv, T, HD, GR).bytes; }

cudaError_t launch_grouped_out_proj_fp4(const Fp4ProjArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const int HD = a.G * a.Kg, GR = a.G * a.R;
  const ProjScratch w = proj_scratch(a.nv, a.T, HD, GR);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  cudaError_t e = launch_fp4_quantize(a.nv, a.o, 1, a.T, HD, HD, a.go, ws + w.o_packed, ws + w.o_scale, s);
  if (e != cudaSuccess) return e;
  Fp4LinearArgs l{};
  l.nv = a.nv;
  l.M = a.T;
  l.N = a.R;
  l.K = a.Kg;
  l.G = a.G;
  l.x_packed = ws + w.o_packed;
  l.x_scale = ws + w.o_scale;
  l.gx = a.go;
  l.w_packed = a.a_packed;
  l.w_scale = a.a_scale;
  l.gw = a.ga;
  l.out_bf16 = 1;
  l.y = ws + w.z;
  l.ldy = GR;
  e = launch_fp4_linear(l, s);
  if (e != cudaSuccess) return e;
  e = launch_fp4_quantize(a.nv, ws + w.z, 1, a.T, GR, GR, a.gz, ws + w.z_packed, ws + w.z_scale, s);
  if (e != cudaSuccess) return e;
  l.N = a.d_model;
  l.K = GR;
  l.G = 1;
  l.x_packed = ws + w.z_packed;
  l.x_scale = ws + w.z_scale;
  l.gx = a.gz;
  l.w_packed = a.b_packed;
  l.w_scale = a.b_scale;
  l.gw = a.gb;
  l.y = a.y;
  l.ldy = a.d_model;
  return launch_fp4_linear(l, s);
}

}  // namespace csa
