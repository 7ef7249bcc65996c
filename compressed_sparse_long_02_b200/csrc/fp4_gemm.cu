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
// axis (kBN a tile), so a single decode token (kBN = 32) streams the weights once and pads
// nothing to 128 rows.  A K slab is 256 elements = 128 bytes a row, one swizzle row.
//
// Roles (512 threads): warp 0 issues the TMA loads (codes, and scale atoms as 512-byte blocks);
// warp 1 owns TMEM and one thread of it issues the MMAs; warps 8-15 write the results (two warps
// per TMEM lane quarter, half of the tile's tokens each; a lane holds one output feature);
// warps 4-7 bring each slab's scales from shared memory to TMEM.  The scales go by
// tcgen05.st: a lane's 16 bytes of an atom are its four columns.  tcgen05.cp from the MMA thread
// runs in order with the MMAs and cost 50-60 cycles per 512-byte atom, 370 (MXFP4) or 650
// (NVFP4) cycles next to a 256 x 256 slab's 512 cycles of MMAs; the stores run beside them.
//
// Pairs (kBN = 256): the two CTAs of a cluster form one tile of 256 features x 256 tokens
// (cta_group::2).  Each loads its own 128 features and half of the tokens, so a slab costs an SM
// 35 KB instead of the 51 KB of a lone 128 x 256 tile (8192 x 4096 x 8192 MXFP4: 198 us with lone
// tiles, 139 with pairs, 98 with the scales and the MMA issue as described here).  The 256
// accumulator columns leave no room for a second accumulator next to the scales: the result warps
// first read the tile into registers, release it, and convert and store while the next tile's MMAs
// run.  A slab then takes 0.38 us, of which 0.27 are MMAs, and the hand-over between two tiles
// 1.5 us without MMAs (7 rounds: 10 of the 98 us).  An SM takes 35 KB a slab, 92 GB/s from L2, but
// that is not what bounds it alone: pairs of 384 tokens (44 KB for 1.5 times the work) measured the
// same, and neither L2 (34 % busy) nor the tensor pipe (56 %) is full.  Back to back for seconds the
// power limit holds the clock near 1.6 GHz and the same product takes 115 us.
//
// Lone CTAs (kBN <= 128): with few tiles the K axis is split over the S CTAs of a cluster.  Each
// CTA sends every other its float32 partial sums of that CTA's tokens (asynchronous stores into
// its shared memory, counted on a barrier), and each adds the S partials of its tokens in rank
// order, so the sum does not depend on timing.  Before it waits for the previous grid, a CTA asks
// for its weights in L2: a hint, which reads nothing, so it may run ahead of whatever wrote them.
//
// Results are float32 or bf16, or (the projection's intermediate) rounded to bf16 and encoded
// again: the scales' blocks run along the features, which a warp's lanes hold.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "fp4.cuh"
#include "internal.h"
#include "mxfp4.cuh"
#include "ptx.cuh"
#include "tmap.h"

namespace csa {
namespace {

constexpr int kTileN = 128;          // output features of a tile (MMA M)
constexpr int kSlabBytes = 128;      // bytes of a row in a K slab: 256 elements
constexpr int kSlab = 2 * kSlabBytes;
constexpr int kThreads = 512;
constexpr int kHintWarp = 2;         // asks for the first tile's weights in L2
constexpr int kSfWarp = 4;           // first of the four scale warps
constexpr int kOutWarp = 8;          // first of the eight result warps

constexpr int kPart = 32;
constexpr uint32_t kPartBytes = kPart * kTileN * 2;  // see part_at

enum Out { kOutF32, kOutBf16, kOutFp4 };

template <bool kNv, int kBN, int kOut>
struct Shape {
  static constexpr bool kPair = kBN == 256;
  static constexpr int kCtas = kPair ? 2 : 1;
  static constexpr int kAtoms = kNv ? 4 : 2;                   // scale atoms of a slab per 128 rows
  static constexpr int kRowBlocks = (kBN + 127) / 128;         // 128-row scale blocks of the tokens
  static constexpr int kRowsX = kBN / kCtas;                   // tokens that a CTA loads
  static constexpr uint32_t kBytesW = kTileN * kSlabBytes;     // 16 KB
  static constexpr uint32_t kBytesX = kRowsX * kSlabBytes;
  static constexpr uint32_t kBytesSf = 512 * kAtoms * (1 + kRowBlocks);
  static constexpr uint32_t kStage = kBytesW + kBytesX + kBytesSf;
  // lone CTAs: float32 partials, all CTAs', of this CTA's tokens; pairs: two parts of each half
  static constexpr uint32_t kRecv = kPair ? (kOut == kOutF32 ? 0 : 4 * kPart * kTileN * 2) : kBN * kTileN * 4;
  // Up to 32 tokens (decode) two CTAs share an SM: the next launch's CTAs set up, and wait for
  // their grid, next to the running ones.
  static constexpr int kMinBlocks = kBN <= 32 ? 2 : 1;
  static constexpr int kFit = static_cast<int>(((kMinBlocks == 2 ? 111u : 225u) * 1024u - kRecv) / kStage);
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStage + kRecv + 512;
  static constexpr int kAcc = kPair ? 1 : 2;                   // accumulators of kBN columns
  static constexpr uint32_t kSfCols = 4 * kAtoms * (1 + kRowBlocks);  // TMEM columns of a slab's scales
  static constexpr uint32_t kColSf = kAcc * kBN;
  static constexpr uint32_t kCols = kColSf + kStages * kSfCols;  // a slot of scales per stage
  static constexpr uint32_t kTmem = kCols <= 128 ? 128 : (kCols <= 256 ? 256 : 512);
  static_assert(kCols <= kTmem && kTmem * kMinBlocks <= 512, "TMEM budget");
  static_assert((kSmem + 1024) * kMinBlocks <= 228 * 1024, "shared memory budget");
  // Registers of a thread after the split, by warpgroup (launched with 65536 / 512 / kMinBlocks each):
  // loads and MMAs, scales, results (two).
  static constexpr int kRegsIssue = kMinBlocks == 1 ? 56 : 40, kRegsSf = kMinBlocks == 1 ? 96 : 56;
  static constexpr int kRegsOut = kMinBlocks == 1 ? 176 : 80;
  static_assert(kRegsIssue + kRegsSf + 2 * kRegsOut <= 4 * (128 / kMinBlocks), "register budget");
};

struct LinearParams {
  int M, N, K, G;
  int n_blocks, m_blocks, tiles, splits;
  int x_atoms, w_atoms;   // scale atoms per row block of X and W
  int x_group_atoms;      // atoms of one group's K columns of X
  int starve;             // kStarve: the barrier, and above 4 bits a bit for each CTA of a cluster in which
  const float* gx;
  const float* gw;
  void* y;
  int64_t ldy;
  int tma_y;              // y has a tensor map (pairs, bf16)
  int vec4;               // rows of y allow stores of 4 features
  uint8_t* z_packed;      // kOutFp4: codes [M, G N / 2], scales, tensor scale
  uint8_t* z_scale;
  const float* gz;
  int z_atoms;
  int32_t* err;
};

// (with the seven tensor maps 1024 bytes of parameters: past that a launch took 0.1 us longer)
static_assert(sizeof(LinearParams) <= 128, "parameters");

template <int kOut>
__device__ __forceinline__ void store_y(void* y, int64_t at, float v) {
  if constexpr (kOut == kOutBf16)
    static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(y)[at] = v;
}

__device__ __forceinline__ float bf16_round(float v) { return __bfloat162float(__float2bfloat16_rn(v)); }

// byte of the scale (token m, block blk) in a blocked layout of n_atoms atoms per row block
__device__ __forceinline__ int64_t scale_at(int m, int blk, int n_atoms) {
  return fp4_atom_offset(m / 128, blk / 4, n_atoms) + (m % 32) * 16 + (m % 128) / 32 * 4 + blk % 4;
}

// A pair's results pass through shared memory in parts of 32 tokens x 128 bf16 features: two
// blocks of 64 features, each [32 tokens][128 bytes] with the 16-byte chunks swizzled by the token
// (SWIZZLE_128B).  The accumulator's 8 x 8 pieces go in transposed (stmatrix), without bank
// conflicts; a TMA store, or the encoder, takes whole rows out.
__device__ __forceinline__ uint32_t part_at(int tok, int chunk) {  // chunk: 8 features, 0..15
  return static_cast<uint32_t>((chunk >> 3) * kPart * 128 + tok * 128 + (((chunk & 7) ^ (tok & 7)) << 4));
}

// The codes of 16 of those features by plain division, from the part's buffer again (out of line:
// extreme scales only).
static __device__ __noinline__ uint2 part_codes_plain(const uint8_t* buf, int tok, int chunk, float T) {
  uint32_t codes[2];
#pragma unroll 1
  for (int q = 0; q < 2; ++q) {
    const uint4 x = *reinterpret_cast<const uint4*>(buf + part_at(tok, chunk + q));
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) bf16x2_floats<true>(w[i], v[2 * i], v[2 * i + 1]);
    codes[q] = nv_codes8_plain(v, T);
  }
  return make_uint2(codes[0], codes[1]);
}

// Encodes 32 consecutive features (feat, a multiple of 32) of one bf16 token of a part's buffer; four
// neighbouring lanes hold the four quarters (b) of 128 features of one token and join their scale bytes.
template <bool kNv>
__device__ __forceinline__ void encode_32(const uint8_t* buf, int tok, int b, bool in, int m, int feat, int n_feat, int n_atoms,
                                          const LinearParams& p, const NvScale& nv) {
  uint4 x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = *reinterpret_cast<const uint4*>(buf + part_at(tok, 4 * b + j));
  const uint32_t w[16] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w,
                          x[2].x, x[2].y, x[2].z, x[2].w, x[3].x, x[3].y, x[3].z, x[3].w};
  uint32_t codes[4], bytes = 0;
  float inv[2], top[2], rcp[2];
  bool plain[2] = {false, false};
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // halves of 16: a block each (NVFP4) or together (MXFP4)
    uint32_t am = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) am = bf16x2_max(am, w[8 * h + i] & 0x7FFF7FFFu);
    top[h] = fmaxf(fmaxf(__uint_as_float(am << 16), __uint_as_float(am & 0xFFFF0000u)), 0.f);
  }
  if constexpr (kNv) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t byte = nv.byte(top[h]);
      bytes |= byte << (8 * h);
      inv[h] = e4m3_value(byte) * nv.g;  // T
      rcp[h] = __frcp_rn(inv[h]);
      plain[h] = inv[h] != 0.f && nv_plain<true>(inv[h], top[h]);
    }
  } else {
    const int E = mx_block_exponent(fmaxf(top[0], top[1]));
    bytes = E + 127;
    inv[0] = inv[1] = mx_pow2_neg(E);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) bf16x2_floats<kNv>(w[4 * q + i], v[2 * i], v[2 * i + 1]);
    codes[q] = kNv ? (inv[q / 2] == 0.f ? 0u : nv_codes8_common<true>(v, inv[q / 2], rcp[q / 2])) : e2m1x8_rn(v, inv[q / 2]);
  }
  const int lane = threadIdx.x & 31;
  if constexpr (kNv) {  // two bytes per lane: lanes 0, 1 hold one atom's four scales, lanes 2, 3 the next's
    bytes <<= 16 * (lane & 1);
    bytes |= __shfl_xor_sync(0xffffffffu, bytes, 1);
  } else {
    bytes <<= 8 * (lane & 3);
    bytes |= __shfl_xor_sync(0xffffffffu, bytes, 1);
    bytes |= __shfl_xor_sync(0xffffffffu, bytes, 2);
  }
  if constexpr (kNv) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (in && plain[h]) {
        const uint2 c = part_codes_plain(buf, tok, 4 * b + 2 * h, inv[h]);
        codes[2 * h] = c.x, codes[2 * h + 1] = c.y;
      }
    }
  }
  if (in) {
    *reinterpret_cast<uint4*>(p.z_packed + (static_cast<int64_t>(m) * n_feat + feat) / 2) =
        make_uint4(codes[0], codes[1], codes[2], codes[3]);
    if (lane % (kNv ? 2 : 4) == 0)
      *reinterpret_cast<uint32_t*>(p.z_scale + scale_at(m, feat / (kNv ? 16 : 32), n_atoms)) = bytes;
  }
}

// Encodes four features (n_feat per row) of one token: a warp holds 128 consecutive features.
template <bool kNv>
__device__ __forceinline__ void encode_row(const float (&o)[4], int m, int feat, int n_feat, int n_atoms,
                                           const LinearParams& p, const NvScale& nv) {
  float x[4], am = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = bf16_round(o[e]);
    am = fmaxf(am, fabsf(x[e]));
  }
  constexpr int kBlk = kNv ? 16 : 32;
#pragma unroll
  for (int d = 1; d < kBlk / 4; d <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, d));
  uint32_t byte, codes;
  if constexpr (kNv) {
    byte = nv.byte(am);
    nv_quotients(x, e4m3_value(byte) * nv.g, am);
    codes = e2m1x2_rn(x[0], x[1]) | e2m1x2_rn(x[2], x[3]) << 8;
  } else {
    const int E = mx_block_exponent(am);
    const float s = mx_pow2_neg(E);
    byte = E + 127;
    codes = e2m1x2_rn(x[0] * s, x[1] * s) | e2m1x2_rn(x[2] * s, x[3] * s) << 8;
  }
  reinterpret_cast<uint16_t*>(p.z_packed)[(static_cast<int64_t>(m) * n_feat + feat) / 4] = static_cast<uint16_t>(codes);
  if (feat % kBlk == 0) p.z_scale[scale_at(m, feat / kBlk, n_atoms)] = static_cast<uint8_t>(byte);
}

// The tensor scales of a product where gx gw is no normal float32: gx gw = pre alpha, pre a power of two
// and alpha normal, so that y = (sum pre) alpha rounds once.  A sum is 0 or in [2^-20, 2^53] (terms are
// multiples of (2^-1 2^-9)^2, at most (6 448)^2, and at most 2^30 of them), so sum pre is exact for pre in
// [2^-100, 2^70]; past either end every result is 0 or infinite as it should be, and a sum of 0 stays 0.
static __device__ __noinline__ float2 wide_scales(float gx, float gw) {
  int ex, ew;
  const float m = frexpf(gx, &ex) * frexpf(gw, &ew);  // in [1/4, 1)
  const int e = ex + ew, ea = max(-124, min(e, 127));
  return make_float2(ldexpf(m, ea), ldexpf(1.f, max(-100, min(e - ea, 70))));
}

// kStarve: a barrier waits for an arrival that never comes, and the limit of a wait is 0.1 s
// (csa_selftest_fp4_give_up).
template <bool kNv, int kBN, int kOut, bool kStarve>
__global__ void __launch_bounds__(kThreads, Shape<kNv, kBN, kOut>::kMinBlocks)
    fp4_linear_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ CUtensorMap tm_xt, const __grid_constant__ CUtensorMap tm_wt,
                      const __grid_constant__ CUtensorMap tm_xs, const __grid_constant__ CUtensorMap tm_ws,
                      const __grid_constant__ CUtensorMap tm_y, const LinearParams p) {
  using S = Shape<kNv, kBN, kOut>;
  constexpr bool kPair = S::kPair;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sW = smem;
  uint8_t* sX = sW + S::kStages * S::kBytesW;
  uint8_t* sSf = sX + S::kStages * S::kBytesX;
  float* recv = reinterpret_cast<float*>(sSf + S::kStages * S::kBytesSf);  // [CTA][token][128 features]
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(recv) + S::kRecv);  // of a pair: the leader's are used
  uint64_t* empty = full + S::kStages;
  uint64_t* sf_full = empty + S::kStages;      // a stage's scales have landed in this CTA's shared memory
  uint64_t* sf_ready = sf_full + S::kStages;   // and are in TMEM (of a pair: the leader's are used)
  uint64_t* acc_full = sf_ready + S::kStages;
  uint64_t* acc_empty = acc_full + S::kAcc;
  uint64_t* recv_full = acc_empty + S::kAcc;
  uint64_t* fin = recv_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(fin + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* loads = abort_flag + 1;  // of a pair: slabs that this CTA loaded, (in the leader) that the other
  volatile int* peer_loads = loads + 1;  // one did, and whether the other one gave up
  volatile int* peer_abort = loads + 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // CTA of the cluster: half of the tile's features in a pair, a share of K otherwise
  const int per_tile = kPair ? 2 : p.splits;
  const int rank = static_cast<int>(blockIdx.x) % per_tile;
  const bool leader = !kPair || rank == 0;
  constexpr long long wait_limit = kStarve ? kWaitLimitCycles / 20 : kWaitLimitCycles;  // cycles that a role waits

  if (threadIdx.x == 0) {
    const int starved = kStarve && (p.starve >> (4 + rank) & 1) ? p.starve & 15 : 0;
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], 1 + (starved == 1));
      mbar_init(&empty[s], 1 + (starved == 2));
      mbar_init(&sf_full[s], 1 + (starved == 3));
      mbar_init(&sf_ready[s], 4 * S::kCtas + (starved == 4));
    }
    for (int b = 0; b < S::kAcc; ++b) {
      mbar_init(&acc_full[b], 1 + (starved == 5));
      mbar_init(&acc_empty[b], 8 * S::kCtas + (starved == 6));
    }
    mbar_init(recv_full, 1 + (starved == 7));
    mbar_init(fin, 1);
    *abort_flag = 0;
    if constexpr (kPair) *peer_abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_x);
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_xs);
    prefetch_tmap(&tm_ws);
  }
  if (warp == 1) {
    if constexpr (kPair) {
      tmem_alloc_pair(tmem_slot, S::kTmem);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, S::kTmem);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if (per_tile > 1) cluster_sync_all();  // every CTA's barriers (and a pair's TMEM) are ready
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int first = static_cast<int>(blockIdx.x) / per_tile, step = static_cast<int>(gridDim.x) / per_tile;
  const int slabs = (p.K + kSlab - 1) / kSlab;
  const int slab0 = kPair ? 0 : static_cast<int>(static_cast<int64_t>(slabs) * rank / p.splits);
  const int slab1 = kPair ? slabs : static_cast<int>(static_cast<int64_t>(slabs) * (rank + 1) / p.splits);
  auto commit = [](uint64_t* bar) {
    if constexpr (kPair)
      tc_commit_pair(bar);
    else
      tc_commit(bar);
  };
  // tile t: features [n0, n0 + 128) of group g (this CTA's), tokens [m0, m0 + kBN); feature blocks
  // run fastest, so the CTAs at work share a few token blocks and all weights of L2
  auto tile = [&](int t, int& n0, int& g, int& m0) {
    const int nb = t % p.n_blocks, mg = t / p.n_blocks;
    n0 = (nb * S::kCtas + (kPair ? rank : 0)) * kTileN;
    g = mg % p.G;
    m0 = mg / p.G * kBN;
  };

  if (warp == kHintWarp && first < p.tiles) {  // the hint: a slab per lane
    int n0, g, m0;
    tile(first, n0, g, m0);
    const int w_row = g * p.N + n0, sl = slab0 + lane;
    if (sl < slab1 && n0 < p.N) {
      tma_prefetch_2d(n0 + kTileN <= p.N ? &tm_w : &tm_wt, sl * kSlabBytes, w_row);
      tma_prefetch_2d(&tm_ws, 0, w_row / 128 * p.w_atoms + sl * S::kAtoms);
    }
  }
  griddep_enter();

  if (warp < kSfWarp) {
    regs_dec<S::kRegsIssue>();
    if (warp == 0) {
      // ---------------------------------------------------------------- loads
      if (lane == 0) {
        int j = 0;
        bool ok = true;
        for (int t = first; ok && t < p.tiles; t += step) {
          int n0, g, m0;
          tile(t, n0, g, m0);
          const int w_row = g * p.N + n0;
          const int x_row = m0 + (kPair ? rank * S::kRowsX : 0);  // a pair's MMA takes half of its tokens from each CTA
          // Only rows that exist are loaded (the maps tm_xt, tm_wt have the boxes of the last rows): rows
          // past the end cost a load more than rows do -- 4096 x 14 x 2048 took 15.4 us with boxes of 128
          // rows of W, 6.4 us with 14.  What the missing rows of shared memory hold reaches only results
          // that are not stored.
          auto rows_of = [](int total, int at, int box) { return max(0, min(box, total - at)); };
          const int w_rows = rows_of(p.N, n0, kTileN), x_rows = rows_of(p.M, x_row, S::kRowsX);
          int rows = w_rows + x_rows;
          if constexpr (kPair) rows += rows_of(p.N, n0 + kTileN, kTileN) + rows_of(p.M, x_row + S::kRowsX, S::kRowsX);  // the leader's count
          const CUtensorMap* map_w = w_rows == kTileN ? &tm_w : &tm_wt;
          const CUtensorMap* map_x = x_rows == S::kRowsX ? &tm_x : &tm_xt;
          const int w_sf = w_row / 128 * p.w_atoms, x_sf = m0 / 128 * p.x_atoms + g * p.x_group_atoms;
          for (int sl = slab0; sl < slab1; ++sl, ++j) {
            const int st = j % S::kStages;
            if (!mbar_wait(&empty[st], ((j / S::kStages) & 1) ^ 1, p.err, abort_flag, wait_limit)) {
              ok = false;
              break;
            }
            // codes past K and scale blocks past the end read as zeros or belong to columns that no MMA step
            // covers, so every slab of a tile counts the same bytes
            const int sf0 = sl * S::kAtoms;
            const uint32_t dw = smem_u32(sW + st * S::kBytesW), dx = smem_u32(sX + st * S::kBytesX);
            const uint32_t ds = smem_u32(sSf + st * S::kBytesSf);
            mbar_arrive_expect_tx(&sf_full[st], S::kBytesSf);
            tma_load_2d(ds, &tm_ws, &sf_full[st], 0, w_sf + sf0);
            for (int rb = 0; rb < S::kRowBlocks; ++rb)
              tma_load_2d(ds + 512 * S::kAtoms * (1 + rb), &tm_xs, &sf_full[st], 0, x_sf + rb * p.x_atoms + sf0);
            if (leader) mbar_arrive_expect_tx(&full[st], rows * kSlabBytes);
            if constexpr (kPair) {
              const uint32_t bar = dsmem_map(&full[st], 0);
              if (w_rows > 0) tma_load_2d_pair(dw, map_w, bar, sl * kSlabBytes, w_row);
              if (x_rows > 0) tma_load_2d_pair(dx, map_x, bar, g * (p.K / 2) + sl * kSlabBytes, x_row);
            } else {
              tma_load_2d(dw, map_w, &full[st], sl * kSlabBytes, w_row);
              tma_load_2d(dx, map_x, &full[st], g * (p.K / 2) + sl * kSlabBytes, x_row);
            }
          }
        }
        // the last loads issued must have landed before shared memory is reused or freed (of a pair: the
        // leader waits for both CTAs' bytes, and the other CTA for the leader at the end); one limit for all
        const long long t_end = clock64() + wait_limit;
        for (int i = std::max(0, j - S::kStages); i < j; ++i) {
          mbar_wait_until(&sf_full[i % S::kStages], (i / S::kStages) & 1, p.err, t_end);
          if (leader) mbar_wait_until(&full[i % S::kStages], (i / S::kStages) & 1, p.err, t_end);
        }
        if constexpr (kPair) {
          *loads = j;
          if (!leader) dsmem_st(dsmem_map(const_cast<int*>(peer_loads), 0), j);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA issuer
      // The whole warp runs the loop and one lane is elected per slab: with a loop inside `lane == 0`
      // the MMAs of a slab left the tensor pipe idle between them (698 against 512 cycles for a
      // pair's slab, measured without loads).
      if (leader) {
        int j = 0, it = 0;
        bool ok = true;
        for (int t = first; ok && t < p.tiles; t += step, ++it) {
          const int buf = it % S::kAcc;
          if (!warp_wait(&acc_empty[buf], ((it / S::kAcc) & 1) ^ 1, p.err, abort_flag, wait_limit)) break;
          tc_fence_after();
          const uint32_t acc = tmem + kBN * buf;
          for (int sl = slab0; sl < slab1; ++sl, ++j) {
            const int st = j % S::kStages;
            const uint32_t ph = (j / S::kStages) & 1;
            if (!warp_wait(&sf_ready[st], ph, p.err, abort_flag, wait_limit) ||
                !warp_wait(&full[st], ph, p.err, abort_flag, wait_limit)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const int n_mma = min(4, (p.K - sl * kSlab + 63) / 64);
            const uint32_t sfw = tmem + S::kColSf + st * S::kSfCols, sfx = sfw + 4 * S::kAtoms;
            const uint32_t a0 = smem_u32(sW + st * S::kBytesW), b0 = smem_u32(sX + st * S::kBytesX);
            auto mma = [&](int kk) {
              const uint64_t da = smem_desc(a0 + 32 * kk, 16, 1024, kSwizzle128B);
              const uint64_t db = smem_desc(b0 + 32 * kk, 16, 1024, kSwizzle128B);
              const uint32_t accumulate = (sl > slab0 || kk > 0) ? 1u : 0u;
              constexpr int kRows = kTileN * S::kCtas;
              if constexpr (kNv) {
                const uint32_t a = sfw + 4 * kk, b = sfx + 4 * S::kRowBlocks * kk;
                if constexpr (kPair)
                  mma_nvf4_pair(acc, da, db, idesc_nvf4(kRows, kBN), accumulate, a, b);
                else
                  mma_nvf4(acc, da, db, idesc_nvf4(kRows, kBN), accumulate, a, b);
              } else {
                const uint32_t id = 2 * (kk & 1);  // the byte of the scale column of this K = 64 step
                const uint32_t a = (sfw + 4 * (kk >> 1)) | (id << 30), b = (sfx + 4 * S::kRowBlocks * (kk >> 1)) | (id << 30);
                if constexpr (kPair)
                  mma_mxf4_pair(acc, da, db, idesc_mxf4(kRows, kBN, id, id), accumulate, a, b);
                else
                  mma_mxf4(acc, da, db, idesc_mxf4(kRows, kBN, id, id), accumulate, a, b);
              }
            };
            if (elect_one()) {
              if (n_mma == 4) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) mma(kk);
              } else {
                for (int kk = 0; kk < n_mma; ++kk) mma(kk);
              }
              commit(&empty[st]);
              if (sl == slab1 - 1) commit(&acc_full[buf]);
            }
            __syncwarp();
          }
        }
        if (elect_one()) {
          commit(fin);  // (of a pair: in both CTAs, after the commits that arrived on the other's barriers)
        }
        __syncwarp();
        mbar_wait_until(fin, 0, p.err, clock64() + wait_limit);
      }
      __syncwarp();
    }
  } else if (warp < kOutWarp) {
    regs_dec<S::kRegsSf>();
    // ---------------------------------------------------------------- scales to TMEM (warps 4-7)
    // slot of a stage: W in columns [0, 4 kAtoms) (4 per atom), then X (per atom 4 per row block).
    // The stage is loaded again only after the MMAs that read the slot, so the slot is free too.
    const uint32_t dst0 = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + S::kColSf;
    const uint32_t ready0 = kPair ? dsmem_map(sf_ready, 0) : 0u;
    int j = 0;
    bool ok = true;
    for (int t = first; ok && t < p.tiles; t += step) {
      int n0, g, m0;
      tile(t, n0, g, m0);
      for (int sl = slab0; sl < slab1; ++sl, ++j) {
        const int st = j % S::kStages;
        if (!warp_wait(&sf_full[st], (j / S::kStages) & 1, p.err, abort_flag, wait_limit)) {
          ok = false;
          break;
        }
        tc_fence_after();  // the slot's last readers, of which the loads' barrier tells
        const uint4* src = reinterpret_cast<const uint4*>(sSf + st * S::kBytesSf) + lane;
        // a tile of 32 or 64 tokens takes its own columns of the row block's four
        constexpr int kUnits = S::kAtoms * (1 + S::kRowBlocks);
        uint32_t r[4 * kUnits];
        const int sub = kBN < 128 ? m0 % 128 / 32 : 0;
#pragma unroll
        for (int a = 0; a < S::kAtoms; ++a) {
#pragma unroll
          for (int b = 0; b <= S::kRowBlocks; ++b) {
            const uint4 u = src[32 * (S::kAtoms * b + a)];
            uint32_t* d = r + (b == 0 ? 4 * a : 4 * (S::kAtoms + S::kRowBlocks * a + b - 1));
            d[0] = u.x, d[1] = u.y, d[2] = u.z, d[3] = u.w;
            if (kBN < 128 && b > 0) {
              d[0] = sub == 0 ? u.x : (sub == 1 ? u.y : (sub == 2 ? u.z : u.w));
              if (kBN == 64) d[1] = sub == 0 ? u.y : u.w;
            }
          }
        }
        const uint32_t dst = dst0 + st * S::kSfCols;
        static_assert(4 * kUnits <= 48 && 4 * kUnits % 8 == 0, "store widths");
        if constexpr (4 * kUnits >= 32) tmem_st32(dst, r);
        if constexpr (4 * kUnits % 32 >= 16) tmem_st16(dst + 4 * kUnits / 32 * 32, r + 4 * kUnits / 32 * 32);
        if constexpr (4 * kUnits % 16 == 8) tmem_st8(dst + 16, r + 16);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kPair)
            mbar_arrive_cluster(ready0 + 8 * st);
          else
            mbar_arrive(&sf_ready[st]);
        }
      }
    }
  } else {
    regs_inc<S::kRegsOut>();
    // ---------------------------------------------------------------- results (warps 8-15)
    const int quarter = warp & 3, half = (warp - kOutWarp) >> 2;
    constexpr int kHalf = kBN / 2;
    const int f = 32 * quarter + lane, c0 = half * kHalf;  // this lane's feature, this warp's first token of a tile
    float alpha = 1.f, pre = 1.f;  // see wide_scales
    if constexpr (kNv) {
      const float gx = p.gx ? __ldg(p.gx) : 1.f, gw = p.gw ? __ldg(p.gw) : 1.f;
      alpha = gx * gw;
      if (!(alpha >= 0x1p-126f && alpha < INFINITY) && gx > 0.f && gw > 0.f && gx < INFINITY && gw < INFINITY) {
        const float2 f = wide_scales(gx, gw);
        alpha = f.x, pre = f.y;
      }
    }
    const bool wide = kNv && pre != 1.f;
    const NvScale nvz(kOut == kOutFp4 && kNv ? __ldg(p.gz) : 1.f);
    const uint32_t acc_done = kPair ? dsmem_map(acc_empty, 0) : 0u;
    if (!kPair && p.splits > 1 && warp == kOutWarp && lane == 0) {  // the bytes this CTA will receive
      int n0, g, m0;
      tile(first, n0, g, m0);
      const int m_valid = min(kBN, p.M - m0), cap = (m_valid + p.splits - 1) / p.splits;
      mbar_arrive_expect_tx(recv_full, max(0, min(cap, m_valid - rank * cap)) * kTileN * 4 * p.splits);
    }
    int it = 0;
    for (int t = first; t < p.tiles; t += step, ++it) {
      const int buf = it % S::kAcc;
      const bool got = warp_wait_sleep(&acc_full[buf], (it / S::kAcc) & 1, p.err, abort_flag, wait_limit);
      // warps that meet at barriers below leave together, whatever each saw (a wait may be given up just as
      // it ends); an unsplit lone CTA's do so there
      if constexpr (kPair && kOut != kOutF32) {
        if (named_bar_or(1 + half, 128, !got)) break;
      } else if (!got && (kPair || p.splits > 1)) {
        break;
      }
      tc_fence_after();
      int n0, g, m0;
      tile(t, n0, g, m0);
      const uint32_t src = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + kBN * buf + c0;
      auto release = [&] {  // all read: the MMA may reuse this accumulator
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kPair)
            mbar_arrive_cluster(acc_done + 8 * buf);
          else
            mbar_arrive(&acc_empty[buf]);
        }
      };
      const int m_valid = min(kBN, p.M - m0), m_left = m_valid - c0;  // tokens of the tile; of this warp's share
      if constexpr (!kPair) {
        // float32 sums to the CTA that writes the token: itself, or over the cluster
        const int cap = (m_valid + p.splits - 1) / p.splits;
#pragma unroll
        for (int c = 0; c < kHalf; c += 16) {
          if (c >= m_left) break;
          uint32_t u[16];
          tmem_ld16(src + c, u);
          tmem_wait_ld();
          if (p.splits == 1) {
#pragma unroll
            for (int i = 0; i < 16; ++i) recv[(c0 + c + i) * kTileN + f] = __uint_as_float(u[i]);
          } else {
            int r = (c0 + c) / cap, i0 = c0 + c - r * cap;  // the token's CTA, its place there
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if (c + i < m_left) st_async_u32(dsmem_map(recv + (rank * cap + i0) * kTileN + f, r), u[i], dsmem_map(recv_full, r));
              if (++i0 == cap) i0 = 0, ++r;
            }
          }
        }
        release();
        if (p.splits == 1 ? named_bar_or(1, 256, !got) : !warp_wait(recv_full, 0, p.err, abort_flag, wait_limit)) break;
        // a warp takes a token at a time: four features per lane, the partials added in rank order
        const int tok0 = p.splits > 1 ? rank * cap : 0, n_tok = p.splits > 1 ? min(cap, m_valid - rank * cap) : m_valid;
        for (int i = warp - kOutWarp; i < n_tok; i += 8) {
          const float* part = recv + i * kTileN + 4 * lane;
          float4 sum = *reinterpret_cast<const float4*>(part);
          for (int r = 1; r < p.splits; ++r) {
            const float4 q = *reinterpret_cast<const float4*>(part + r * cap * kTileN);
            sum.x += q.x, sum.y += q.y, sum.z += q.z, sum.w += q.w;
          }
          if (wide) sum.x *= pre, sum.y *= pre, sum.z *= pre, sum.w *= pre;
          const float o[4] = {sum.x * alpha, sum.y * alpha, sum.z * alpha, sum.w * alpha};
          const int m = m0 + tok0 + i, n = n0 + 4 * lane;
          const int64_t at = static_cast<int64_t>(m) * p.ldy + static_cast<int64_t>(g) * p.N + n;
          if constexpr (kOut == kOutFp4) {
            encode_row<kNv>(o, m, g * p.N + n, p.G * p.N, p.z_atoms, p, nvz);
          } else if (p.vec4 && n + 3 < p.N) {
            if constexpr (kOut == kOutBf16)
              *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + at) = make_uint2(fp4_bf16x2(o[0], o[1]), fp4_bf16x2(o[2], o[3]));
            else
              *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) = make_float4(o[0], o[1], o[2], o[3]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (n + e < p.N) store_y<kOut>(p.y, at + e, o[e]);
          }
        }
        if (p.splits == 1) named_bar_sync(1, 256);  // the buffer is free for the next tile
      } else if constexpr (kOut == kOutF32) {
        const int n = n0 + f;
        float* y = static_cast<float*>(p.y) + static_cast<int64_t>(m0 + c0) * p.ldy + static_cast<int64_t>(g) * p.N + n;
        uint32_t v[kHalf];
#pragma unroll
        for (int c = 0; c < kHalf; c += 16) tmem_ld16(src + c, v + c);
        tmem_wait_ld();
        release();
        if (wide) {
#pragma unroll
          for (int i = 0; i < kHalf; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * pre);
        }
        if (n < p.N) {
#pragma unroll
          for (int i = 0; i < kHalf; ++i) {
            if (i < m_left) *y = __uint_as_float(v[i]) * alpha;
            y += p.ldy;
          }
        }
      } else {
        // the warp's whole share rounded to bf16 in registers: 8 x 8 pieces, v[i][m] of tokens 8i.. and
        // features 8m.., which leave part by part while the next tile runs
        uint32_t v[kHalf / 8][4];
#pragma unroll
        for (int c = 0; c < kHalf; c += 32) {
          uint32_t u[2][16];
          tmem_ld_16x256b_x4(src + c, u[0]);
          tmem_ld_16x256b_x4(src + (16u << 16) + c, u[1]);
          tmem_wait_ld();
          if (wide) {
#pragma unroll
            for (int i = 0; i < 32; ++i) u[i / 16][i % 16] = __float_as_uint(__uint_as_float(u[i / 16][i % 16]) * pre);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int m = 0; m < 4; ++m)
              v[c / 8 + i][m] = fp4_bf16x2(__uint_as_float(u[m / 2][4 * i + 2 * (m & 1)]) * alpha,
                                           __uint_as_float(u[m / 2][4 * i + 2 * (m & 1) + 1]) * alpha);
          }
        }
        release();
        // the four warps of this half alternate between its two part buffers, one barrier a part: who
        // passes the next part's barrier has left this one's buffer
        const int id = quarter * 32 + lane;
#pragma unroll
        for (int part = 0; part < kHalf / kPart; ++part) {
          uint8_t* buf_z = reinterpret_cast<uint8_t*>(recv) + (2 * half + (part & 1)) * kPartBytes;
#pragma unroll
          for (int i = 0; i < kPart / 8; ++i) {
            const uint32_t* q = v[part * (kPart / 8) + i];
            stmatrix_x4_trans(smem_u32(buf_z) + part_at(8 * i + (lane & 7), 4 * quarter + (lane >> 3)), q[0], q[1], q[2], q[3]);
          }
          const int left = m_left - part * kPart, m = m0 + c0 + part * kPart;  // tokens of this part
          if constexpr (kOut == kOutFp4) {
            named_bar_sync(1 + half, 128);
            const int tok = id / 4, b = id % 4;
            encode_32<kNv>(buf_z, tok, b, tok < left && n0 < p.N, m + tok, g * p.N + n0 + 32 * b, p.G * p.N, p.z_atoms, p, nvz);
          } else if (p.tma_y) {
            fence_proxy_async_smem();
            if (id == 0) bulk_wait_read();  // the other buffer's store has read it
            named_bar_sync(1 + half, 128);
            if (id == 0 && left > 0) {
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (n0 + 64 * h < p.N) tma_store_2d(&tm_y, smem_u32(buf_z) + h * kPart * 128, g * p.N + n0 + 64 * h, m);
              bulk_commit();
            }
          } else {  // rows that no tensor map can describe: a token per warp at a time
            named_bar_sync(1 + half, 128);
            uint16_t* y = static_cast<uint16_t*>(p.y) + static_cast<int64_t>(m) * p.ldy + static_cast<int64_t>(g) * p.N + n0;
#pragma unroll
            for (int k = 0; k < kPart / 4; ++k) {
              const int tok = quarter + 4 * k;
              if (tok >= left) break;
              uint16_t* row = y + tok * p.ldy;
              if (p.vec4) {
                if (n0 + 4 * lane < p.N)
                  reinterpret_cast<uint2*>(row)[lane] = *reinterpret_cast<const uint2*>(buf_z + part_at(tok, lane >> 1) + 8 * (lane & 1));
              } else {
#pragma unroll
                for (int e = lane; e < kTileN; e += 32)
                  if (n0 + e < p.N) row[e] = *reinterpret_cast<const uint16_t*>(buf_z + part_at(tok, e >> 3) + 2 * (e & 7));
              }
            }
          }
        }
      }
    }
    if constexpr (kPair && kOut == kOutBf16) {
      if (quarter == 0 && lane == 0) bulk_wait();  // nothing may read this CTA's shared memory after it is gone
    }
  }

  // no CTA leaves before every CTA of its cluster has sent its partials
  if (!kPair && p.splits > 1) {
    __syncwarp();
    cluster_arrive_relaxed();
    cluster_wait();
  }
  tc_fence_before();
  __syncthreads();
  // nor, having given up, while those sent to it may be on their way
  if (!kPair && p.splits > 1 && warp == kOutWarp && *abort_flag) mbar_wait_until(recv_full, 0, p.err, clock64() + wait_limit);
  if constexpr (kPair) {
    if (warp == 1 && !leader) {
      mbar_wait_until(fin, 0, p.err, clock64() + wait_limit);
      __syncwarp();
    }
    if (threadIdx.x == 0 && *abort_flag) dsmem_st(dsmem_map(const_cast<int*>(peer_abort), rank ^ 1), 1);
    __syncwarp();
    cluster_sync_all();  // neither CTA leaves while the other's MMAs or loads use it
    if (*abort_flag || *peer_abort) {
      // the other CTA may have gone further than the leader and loaded slabs whose bytes the leader never
      // announced (at most a ring of them): it does so now, and waits for them
      if (leader && threadIdx.x == 0) {
        const int j0 = *loads, j1 = *peer_loads;
        for (int j = j0; j < j1; ++j) {
          int n0, g, m0;
          tile(first + j / slabs * step, n0, g, m0);
          const int rows = max(0, min(kTileN, p.N - n0 - kTileN)) + max(0, min(S::kRowsX, p.M - m0 - S::kRowsX));
          mbar_arrive_expect_tx(&full[j % S::kStages], rows * kSlabBytes);
        }
        const long long t_end = clock64() + wait_limit;
        for (int j = j0; j < j1; ++j) mbar_wait_until(&full[j % S::kStages], (j / S::kStages) & 1, p.err, t_end);
      }
      __syncwarp();
      cluster_sync_all();
    }
  }
  if (warp == 1) {
    tc_fence_after();
    if constexpr (kPair)
      tmem_dealloc_pair(tmem, S::kTmem);
    else
      tmem_dealloc(tmem, S::kTmem);
  }
}

// Clusters of `size` CTAs that the device holds at once; fewer than its SMs would give, since a
// cluster stays within one GPC.
template <typename K>
int resident_clusters(K k, size_t smem, int size) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(num_sms() / size * size));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  return cudaOccupancyMaxActiveClusters(&n, k, &cfg) == cudaSuccess && n > 0 ? n : num_sms() / size;
}

template <bool kNv, int kBN, int kOut, bool kStarve>
cudaError_t launch_tile(const Fp4LinearArgs& a, LinearParams& p, int splits, cudaStream_t s) {
  using Sh = Shape<kNv, kBN, kOut>;
  static int smem_set[64], resident[64];  // pairs: what runs at once, per device
  CUtensorMap tm_x, tm_w, tm_xt = {}, tm_wt = {}, tm_xs, tm_ws, tm_y = {};
  const uint64_t xb = static_cast<uint64_t>(a.G) * a.K / 2, wb = a.K / 2, w_rows = static_cast<uint64_t>(a.G) * a.N;
  const uint32_t x_tail = a.M % Sh::kRowsX, w_tail = a.N % kTileN;  // (groups are whole tiles)
  if (!encode_2d_u8(&tm_x, a.x_packed, xb, a.M, kSlabBytes, Sh::kRowsX, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d_u8(&tm_w, a.w_packed, wb, w_rows, kSlabBytes, kTileN, CU_TENSOR_MAP_SWIZZLE_128B) ||
      (x_tail != 0 && !encode_2d_u8(&tm_xt, a.x_packed, xb, a.M, kSlabBytes, x_tail, CU_TENSOR_MAP_SWIZZLE_128B)) ||
      (w_tail != 0 && !encode_2d_u8(&tm_wt, a.w_packed, wb, w_rows, kSlabBytes, w_tail, CU_TENSOR_MAP_SWIZZLE_128B)) ||
      !encode_blocks_512(&tm_xs, a.x_scale, static_cast<uint64_t>((a.M + 127) / 128) * p.x_atoms, Sh::kAtoms) ||
      !encode_blocks_512(&tm_ws, a.w_scale, (w_rows + 127) / 128 * p.w_atoms, Sh::kAtoms))
    return cudaErrorInvalidValue;
  if (Sh::kPair && kOut == kOutBf16 && a.N % 8 == 0 && a.ldy % 8 == 0)
    p.tma_y = encode_2d_bf16(&tm_y, a.y, w_rows, a.M, a.ldy, kPart);
  p.m_blocks = (a.M + kBN - 1) / kBN;
  p.n_blocks = (a.N + kTileN * Sh::kCtas - 1) / (kTileN * Sh::kCtas);
  const int64_t tiles = static_cast<int64_t>(p.m_blocks) * p.n_blocks * a.G;
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
  p.tiles = static_cast<int>(tiles);
  auto k = fp4_linear_kernel<kNv, kBN, kOut, kStarve>;
  const cudaError_t e = set_dyn_smem(reinterpret_cast<const void*>(k), Sh::kSmem, smem_set);
  if (e != cudaSuccess) return e;
  const dim3 block(kThreads);
  if constexpr (Sh::kPair) {
    p.splits = 1;
    int dev = 0;
    cudaGetDevice(&dev);  // 0..63: set_dyn_smem accepted it
    if (resident[dev] == 0) resident[dev] = resident_clusters(k, Sh::kSmem, 2);
    const int64_t n = std::min<int64_t>(tiles, resident[dev]);
    return launch_pdl_cluster(k, dim3(static_cast<unsigned>(2 * n)), block, Sh::kSmem, 2, s, tm_x, tm_w, tm_xt, tm_wt, tm_xs, tm_ws, tm_y, p);
  } else {
    p.splits = splits;
    const int64_t clusters = splits > 1 ? tiles : std::min<int64_t>(tiles, num_sms() * Sh::kMinBlocks);
    const dim3 grid(static_cast<unsigned>(clusters * p.splits));
    if (p.splits == 1) return launch_pdl(k, grid, block, Sh::kSmem, s, tm_x, tm_w, tm_xt, tm_wt, tm_xs, tm_ws, tm_y, p);
    return launch_pdl_cluster(k, grid, block, Sh::kSmem, p.splits, s, tm_x, tm_w, tm_xt, tm_wt, tm_xs, tm_ws, tm_y, p);
  }
}

// Tokens per tile and CTAs per tile (a split of K), by the time that each choice would take in
// nanoseconds beyond what all have in common.  Measured on one B200 (us; 32 / 64 / 128 tokens a
// tile at their best splits, and pairs): 1 x 4096 x 8192 6.5 / 7.6 / 8.7 / 15; 64 x 4096 x 8192
// 9.5 / 9.1 / 10 / 15; 256 x 4096 x 8192 19 / 17 / 14.5 / 16; 512 x 4096 x 8192 32 / 29 / 18.5 /
// 16.4; 600 x 256 x 512, 4 groups, 4.5 / 4.5 / 5.4 / 5.6.  The terms, from the same runs:
//   a slab of a lone CTA 370, 400, 430 by its width (what one SM loads), 480 with two on an SM;
//   a slab of a pair 380, and 1500 for the hand-over between tiles (2500 where rows of y have no
//   tensor map);
//   a split 400 plus 30 a token for the exchanged sums (35 at 64 and 128 tokens, and 400 for a
//   set-up that no launch before it hides; twice the 30 and 1500 on a shared SM);
//   unsplit results 10 a token.
// In batch-invariant mode K is never split, so a row's sums run over K in one order whatever the
// number of rows; few rows pay for it (x 4096 x 8192 MXFP4: 1 token 14.4 us for 6.5, 32 tokens 14.9
// for 7.1, 128 tokens 15.3 for 11.1, 512 the same).
struct Choice {
  int tokens, splits;
};
// resident[wide][i]: clusters of 2^i lone CTAs that run at once, 32 tokens a tile or wider
Choice choose(const Fp4LinearArgs& a, const int (&resident)[2][4]) {
  const int64_t slabs = (a.K + kSlab - 1) / kSlab, sms = num_sms();
  const int64_t rows = static_cast<int64_t>(a.G) * ((a.N + kTileN - 1) / kTileN);
  const int64_t pairs = static_cast<int64_t>(a.G) * ((a.N + 2 * kTileN - 1) / (2 * kTileN)) * ((a.M + 255) / 256);
  const bool tma_y = a.z_packed != nullptr || (a.out_bf16 && a.N % 8 == 0 && a.ldy % 8 == 0);
  Choice best{256, 1};
  int64_t cost = (pairs + sms / 2 - 1) / (sms / 2) * (slabs * 380 + (tma_y ? 1500 : 2500));
  for (int i = 0; i < 3; ++i) {
    const int bn = 32 << i;
    const int64_t tiles = rows * ((a.M + bn - 1) / bn), tok = std::min(a.M, bn);
    for (int j = 0; j < (batch_invariant() ? 1 : 4) && (1 << j) <= slabs; ++j) {
      const int64_t ctas = tiles << j, shared = bn == 32 && ctas > sms ? 1 : 0, room = resident[i > 0][j];
      if (j > 0 && tiles > room) break;
      const int64_t slab = bn == 32 ? (shared ? 480 : 370) : (bn == 64 ? 400 : 430);
      const int64_t ends = j == 0 ? 10 * (1 + shared) * tok
                                  : 400 + (bn == 32 ? 30 * (1 + shared) * tok + 1500 * shared : 35 * tok + 400);
      const int64_t c = (tiles + room - 1) / room * (((slabs + (1 << j) - 1) >> j) * slab + ends);
      if (c < cost) cost = c, best = Choice{bn, 1 << j};
    }
  }
  return best;
}

// The table of choose() for a format and a kind of result, asked for once per device.
template <bool kNv, int kOut>
cudaError_t lone_residents(const int (**out)[2][4]) {
  static int table[64][2][4];
  static int smem_set[2][64];
  int dev = 0;
  const cudaError_t g = cudaGetDevice(&dev);
  if (g != cudaSuccess) return g;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  *out = &table[dev];
  if (table[dev][1][3] != 0) return cudaSuccess;
  const auto narrow = fp4_linear_kernel<kNv, 32, kOut, false>, wide = fp4_linear_kernel<kNv, 128, kOut, false>;
  constexpr size_t narrow_smem = Shape<kNv, 32, kOut>::kSmem, wide_smem = Shape<kNv, 128, kOut>::kSmem;
  cudaError_t e = set_dyn_smem(reinterpret_cast<const void*>(narrow), narrow_smem, smem_set[0]);
  if (e == cudaSuccess) e = set_dyn_smem(reinterpret_cast<const void*>(wide), wide_smem, smem_set[1]);
  if (e != cudaSuccess) return e;
  for (int i = 0; i < 4; ++i) {
    table[dev][0][i] = resident_clusters(narrow, narrow_smem, 1 << i);
    table[dev][1][i] = resident_clusters(wide, wide_smem, 1 << i);
  }
  return cudaSuccess;
}

template <bool kNv, int kOut, bool kStarve = false>
cudaError_t launch_shape(const Fp4LinearArgs& a, LinearParams& p, cudaStream_t s) {
  const int(*resident)[2][4] = nullptr;
  const cudaError_t e = lone_residents<kNv, kOut>(&resident);
  if (e != cudaSuccess) return e;
  const Choice c = choose(a, *resident);
  switch (c.tokens) {
    case 32: return launch_tile<kNv, 32, kOut, kStarve>(a, p, c.splits, s);
    case 64: return launch_tile<kNv, 64, kOut, kStarve>(a, p, c.splits, s);
    case 128: return launch_tile<kNv, 128, kOut, kStarve>(a, p, c.splits, s);
    default: return launch_tile<kNv, 256, kOut, kStarve>(a, p, 1, s);
  }
}

}  // namespace

cudaError_t launch_fp4_linear(const Fp4LinearArgs& a, cudaStream_t s) {
  if (a.M == 0 || a.N == 0) return cudaSuccess;
  LinearParams p{};
  p.M = a.M;
  p.N = a.N;
  p.K = a.K;
  p.G = a.G;
  p.x_atoms = fp4_atoms(a.nv, a.G * a.K);
  p.w_atoms = fp4_atoms(a.nv, a.K);
  p.x_group_atoms = a.G > 1 ? p.w_atoms : 0;
  p.gx = a.gx;
  p.gw = a.gw;
  p.y = a.y;
  p.ldy = a.ldy;
  p.vec4 = a.N % 4 == 0 && a.ldy % 4 == 0;
  p.z_packed = a.z_packed;
  p.z_scale = a.z_scale;
  p.gz = a.gz;
  p.z_atoms = fp4_atoms(a.nv, a.G * a.N);
  p.err = device_error_word();
  if (p.err == nullptr) return cudaErrorUnknown;
  if (a.starve != 0) {
    p.starve = a.starve | a.starve_ranks << 4;
    return a.nv ? launch_shape<true, kOutF32, true>(a, p, s) : launch_shape<false, kOutBf16, true>(a, p, s);
  }
  if (a.z_packed != nullptr) return a.nv ? launch_shape<true, kOutFp4>(a, p, s) : launch_shape<false, kOutFp4>(a, p, s);
  if (a.nv) return a.out_bf16 ? launch_shape<true, kOutBf16>(a, p, s) : launch_shape<true, kOutF32>(a, p, s);
  return a.out_bf16 ? launch_shape<false, kOutBf16>(a, p, s) : launch_shape<false, kOutF32>(a, p, s);
}

// ------------------------------------------------------------------ grouped output projection
// Scratch of the projection, 256-byte aligned pieces: the codes and scales of o and of z (the
// first product encodes z as it writes it).
namespace {
struct ProjScratch {
  size_t o_packed, o_scale, z_packed, z_scale, bytes;
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
  l.z_packed = ws + w.z_packed;
  l.z_scale = ws + w.z_scale;
  l.gz = a.gz;
  e = launch_fp4_linear(l, s);
  if (e != cudaSuccess) return e;
  l.z_packed = l.z_scale = nullptr;
  l.out_bf16 = 1;
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
