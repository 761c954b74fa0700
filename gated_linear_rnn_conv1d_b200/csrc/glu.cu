// The gated feed-forward block ("Griffin：将门控线性循环与局部注意力混合以实现高效的语言模型",
// §MLP块 (gated MLP, Fig. 2(b))) without its down projection, and its backward:
//     g = x W_gᵀ,  u = x W_uᵀ,  h = act(g) ⊙ u,              x [N][D], W_g, W_u [H][D]
//     dg = dh ⊙ u ⊙ act'(g),  du = dh ⊙ act(g)               (g and u formed again from x)
//     dx = dg W_g + du W_u,   dW_g = dgᵀ x,  dW_u = duᵀ x.
// Five products of 2·N·D·H operations or six halves of them: the tensor cores bound every part,
// so the elementwise work rides in the products' epilogues and g, u are never stored.
//
// One kernel shape: persistent CTA pairs (cta_group::2) on 256 × 256 output tiles, as the gate
// GEMM's: warp 0 loads by TMA, warp 1 of the leader issues the MMAs, eight warps of each CTA
// empty one accumulator while the next tile's MMAs fill the other. Four modes of it:
//   GLU_FWD   h: rank 0 stages 128 rows of W_g, rank 1 the same 128 rows of W_u, so a tile holds
//             g in columns 0–127 and u of the same channels in 128–255.
//   GLU_GRAD  the same products; the epilogue reads dh and writes dg, du (and h when asked for).
//   GLU_DX    dx: [dg | du]·[W_g; W_u], the weights read in place as an MN-major operand; k runs
//             over dg's channels, then over du's.
//   GLU_DW    dW_g and dW_u: dgᵀx and duᵀx, both operands MN-major in place, k over the tokens.
// Ragged sizes need no code in the loops: TMA fills what lies outside a matrix with zeros.
#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>

#include "act_math.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace rglru {
namespace {

constexpr int BK = 64;  // 64 bf16 = one 128-byte swizzle row
constexpr int kStages = 6;
constexpr int kABytes = 128 * BK * 2;  // this CTA's 128 rows of A
constexpr int kBBytes = 128 * BK * 2;  // this CTA's half of the B tile
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kSmem = kStages * kStageBytes + 1024;
constexpr int kTmemCols = 512;  // two 256-column accumulators
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr uint32_t kIdesc = umma_idesc_bf16_f32(256, 256);
// Output tiles are taken in bands of kBand tile rows, column by column: the 74 pairs at work at
// a time then cover about 8 × 9 tiles, whose operands (17 · 256 rows of k) stay in L2 between them.
constexpr int kBand = 8;

enum GluMode { GLU_FWD = 0, GLU_GRAD = 1, GLU_DX = 2, GLU_DW = 3 };

struct GluGemmArgs {
  int64_t M;           // output rows: N tokens, or H channels (GLU_DW)
  int N;               // output columns: H channels (GLU_FWD, GLU_GRAD) or D
  int tiles_m, tiles_n;
  int tiles_half;      // GLU_DW: tile rows of dW_g (dW_u's follow)
  int kb_half;         // GLU_DX: k-blocks of dg (du's follow)
  int k_blocks;
  __nv_bfloat16* out0;        // h | dg | dx | dW_g
  __nv_bfloat16* out1;        // – | du | –  | dW_u
  __nv_bfloat16* h;           // GLU_GRAD: h, or null
  const __nv_bfloat16* dh;    // GLU_GRAD
};

__device__ __forceinline__ void tile_of(const GluGemmArgs& a, int tile, int& m, int& n) {
  const int band = tile / (kBand * a.tiles_n);
  const int r = tile - band * kBand * a.tiles_n;
  const int rows = min(kBand, a.tiles_m - band * kBand);
  n = r / rows;
  m = band * kBand + r - n * rows;
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

template <int MODE, int ACT>
__global__ void __launch_bounds__(kThreads, 1)
    glu_gemm_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1,
                    const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1,
                    const GluGemmArgs args, unsigned* status) {
  constexpr bool kAMN = MODE == GLU_DW;                    // A MN-major
  constexpr bool kBMN = MODE == GLU_DX || MODE == GLU_DW;  // B MN-major
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[kStages];
  __shared__ __align__(8) uint64_t empty_bar[kStages];
  __shared__ __align__(8) uint64_t tfull_bar[2];
  __shared__ __align__(8) uint64_t tempty_bar[2];
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_s;

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster = blockIdx.x / 2;
  const int n_clusters = gridDim.x / 2;
  const int num_tiles = args.tiles_m * args.tiles_n;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full_bar[i], 1);
      mbar_init(&empty_bar[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull_bar[i], 1);
      mbar_init(&tempty_bar[i], 2 * kEpiWarps);  // the epilogue warps of both CTAs
    }
    mbar_init(&drain_bar, 1);
    abort_s = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA0);
    tma_prefetch_desc(&tmB0);
    if (MODE != GLU_DW) tma_prefetch_desc(&tmB1);
    if (MODE == GLU_DX || MODE == GLU_DW) tma_prefetch_desc(&tmA1);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_s)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  cluster_sync_all();  // both CTAs' barriers initialised and TMEM allocated
  tc_fence_after();
  pdl_wait();  // what this kernel reads or overwrites is settled from here on
  pdl_launch_dependents();
  const uint32_t tmem_base = tmem_base_s;
  const uint32_t leader_full0 = mapa_rank(smem_u32(&full_bar[0]), 0);

  if (warp == 0) {
    // ---------------- TMA producer (both CTAs) ----------------
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = cluster; tile < num_tiles && ok; tile += n_clusters) {
        int m, n;
        tile_of(args, tile, m, n);
        const bool second_m = MODE == GLU_DW && m >= args.tiles_half;
        const int arow = (m - (second_m ? args.tiles_half : 0)) * 256 + (int)rank * 128;
        const int bcol = MODE == GLU_FWD || MODE == GLU_GRAD ? n * 128 : n * 256 + (int)rank * 128;
        for (int kb = 0; kb < args.k_blocks; ++kb) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1, &abort_s)) { ok = false; break; }
          uint8_t* sa = smem + stage * kStageBytes;
          uint8_t* sb = sa + kABytes;
          const uint32_t lbar = leader_full0 + stage * 8;
          if (leader) mbar_arrive_expect_tx(&full_bar[stage], 2 * kStageBytes);
          const bool second_k = MODE == GLU_DX && kb >= args.kb_half;
          const int kc = (kb - (second_k ? args.kb_half : 0)) * BK;
          const CUtensorMap* ma = second_m || second_k ? &tmA1 : &tmA0;
          if constexpr (kAMN) {  // 128 columns as two boxes of 64 columns × BK rows
            tma_load_2d_2sm(sa, ma, lbar, arow, kc);
            tma_load_2d_2sm(sa + kABytes / 2, ma, lbar, arow + 64, kc);
          } else {
            tma_load_2d_2sm(sa, ma, lbar, kc, arow);
          }
          if constexpr (kBMN) {
            const CUtensorMap* mb = second_k ? &tmB1 : &tmB0;
            tma_load_2d_2sm(sb, mb, lbar, bcol, kc);
            tma_load_2d_2sm(sb + kBBytes / 2, mb, lbar, bcol + 64, kc);
          } else {
            tma_load_2d_2sm(sb, leader ? &tmB0 : &tmB1, lbar, kc, bcol);
          }
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
      }
      if (!ok) { abort_s = 1; atomicOr(status, kStatusTimeout); }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (leader CTA only) ----------------
    if (leader && lane == 0) {
      constexpr uint32_t idesc = kIdesc | (kAMN ? kIdescAMN : 0u) | (kBMN ? kIdescBMN : 0u);
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int tile = cluster; tile < num_tiles && ok; tile += n_clusters) {
        if (!mbar_wait(&tempty_bar[acc], acc_phase ^ 1, &abort_s)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * 256;
        for (int kb = 0; kb < args.k_blocks; ++kb) {
          if (!mbar_wait(&full_bar[stage], phase, &abort_s)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(smem + stage * kStageBytes);
          const uint32_t b_addr = a_addr + kABytes;
          // one MMA takes 16 of k: 32 bytes along K-major rows, 16 rows of 128 B of an MN-major box
#pragma unroll
          for (int k = 0; k < BK / 16; ++k)
            umma_f16_2sm(d_tmem,
                         kAMN ? umma_desc_sw128_mn(a_addr + k * 2048, kABytes / 2) : umma_desc_sw128(a_addr + k * 32),
                         kBMN ? umma_desc_sw128_mn(b_addr + k * 2048, kBBytes / 2) : umma_desc_sw128(b_addr + k * 32),
                         idesc, (kb | k) != 0 ? 1u : 0u);
          umma_commit_2sm_both(&empty_bar[stage]);
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
        umma_commit_2sm_both(&tfull_bar[acc]);
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
      if (!ok) { abort_s = 1; atomicOr(status, kStatusTimeout); }
      // every MMA issued here has completed before TMEM is freed
      asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                       smem_u32(&drain_bar))
                   : "memory");
      volatile int never = 0;
      (void)mbar_wait(&drain_bar, 0, &never);
    }
  } else {
    // ---------------- epilogue warps (both CTAs) ----------------
    // warp w empties TMEM lanes 32·(w mod 4) … (one output row a thread) and one half of the
    // columns: 64 channels' g and u, or 128 plain columns.
    const int quarter = warp & 3;
    const int half = (warp - 2) / 4;
    const uint32_t leader_tempty0 = mapa_rank(smem_u32(&tempty_bar[0]), 0);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int tile = cluster; tile < num_tiles; tile += n_clusters) {
      int m, n;
      tile_of(args, tile, m, n);
      const bool second_m = MODE == GLU_DW && m >= args.tiles_half;
      const int64_t row = (int64_t)(m - (second_m ? args.tiles_half : 0)) * 256 + rank * 128 + quarter * 32 + lane;
      const bool row_ok = row < args.M;
      constexpr bool kGated = MODE == GLU_FWD || MODE == GLU_GRAD;
      const int col0 = kGated ? n * 128 + half * 64 : n * 256 + half * 128;
      const int64_t base = row * args.N + col0;
      // dh of this thread's row, loaded before the accumulator is ready
      [[maybe_unused]] uint4 dhq[MODE == GLU_GRAD ? 8 : 1];
      if constexpr (MODE == GLU_GRAD) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          dhq[q] = row_ok && col0 + 8 * q < args.N ? __ldg(reinterpret_cast<const uint4*>(args.dh + base) + q)
                                                   : make_uint4(0u, 0u, 0u, 0u);
      }
      if (!mbar_wait(&tfull_bar[acc], acc_phase, &abort_s)) {
        abort_s = 1;
        atomicOr(status, kStatusTimeout);
        break;
      }
      tc_fence_after();
      const uint32_t t_row = tmem_base + ((uint32_t)(quarter * 32) << 16) + acc * 256;
      // four pairs of 16 columns; the next pair's TMEM loads are in flight while one is worked on
      const uint32_t ta = t_row + half * (kGated ? 64 : 128), tb = ta + (kGated ? 128 : 16);
      constexpr int kStep = kGated ? 16 : 32;
      uint32_t ra[2][16], rb[2][16];
      tmem_ld_x16(ta, ra[0]);
      tmem_ld_x16(tb, rb[0]);
      tmem_ld_wait16(ra[0], rb[0]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int cur = k & 1;
        if (k + 1 < 4) {
          tmem_ld_x16(ta + (k + 1) * kStep, ra[cur ^ 1]);
          tmem_ld_x16(tb + (k + 1) * kStep, rb[cur ^ 1]);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {  // eight columns of each, all inside the matrix or all outside
          const int c = col0 + k * kStep + q * 8;
          if constexpr (kGated) {
            float o0[8];
            [[maybe_unused]] float o1[8], o2[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float g = __uint_as_float(ra[cur][q * 8 + j]), u = __uint_as_float(rb[cur][q * 8 + j]);
              float slope = 0.0f;
              const float a = g * act_gate<ACT, MODE == GLU_GRAD>(g, slope);
              if constexpr (MODE == GLU_FWD) {
                o0[j] = a * u;
              } else {
                const uint4 d4 = dhq[2 * k + q];
                const uint32_t w = j < 2 ? d4.x : j < 4 ? d4.y : j < 6 ? d4.z : d4.w;
                const float d = j % 2 == 0 ? bf16lo(w) : bf16hi(w);
                // dg and du are rounded to bf16, the operands of the next products: half a step
                // of 2^-8 each, as much as the rounding of dx and dW themselves
                o0[j] = d * u * slope;
                o1[j] = d * a;
                o2[j] = a * u;
              }
            }
            if (row_ok && c < args.N) {
              const int64_t at = base + k * kStep + q * 8;
              *reinterpret_cast<uint4*>(args.out0 + at) = pack8(o0);
              if constexpr (MODE == GLU_GRAD) {
                *reinterpret_cast<uint4*>(args.out1 + at) = pack8(o1);
                if (args.h != nullptr) *reinterpret_cast<uint4*>(args.h + at) = pack8(o2);
              }
            }
          } else {
            __nv_bfloat16* out = second_m ? args.out1 : args.out0;
            float v[8], w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              v[j] = __uint_as_float(ra[cur][q * 8 + j]);
              w[j] = __uint_as_float(rb[cur][q * 8 + j]);
            }
            const int64_t at = base + k * kStep + q * 8;
            if (row_ok && c < args.N) *reinterpret_cast<uint4*>(out + at) = pack8(v);
            if (row_ok && c + 16 < args.N) *reinterpret_cast<uint4*>(out + at + 16) = pack8(w);
          }
        }
        if (k + 1 < 4) tmem_ld_wait16(ra[cur ^ 1], rb[cur ^ 1]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(leader_tempty0 + acc * 8);
      if (++acc == 2) { acc = 0; acc_phase ^= 1; }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the peer's shared memory stays valid until the leader's MMAs are done
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols)
                 : "memory");
  }
}

template <int MODE, int ACT>
cudaError_t launch_mode(const CUtensorMap& a0, const CUtensorMap& a1, const CUtensorMap& b0, const CUtensorMap& b1,
                        const GluGemmArgs& args, unsigned* status, cudaStream_t s) {
  auto kern = glu_gemm_kernel<MODE, ACT>;
  static bool attr_set[64] = {};  // idempotent: a race sets it twice
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  const int64_t tiles = (int64_t)args.tiles_m * args.tiles_n;
  if (tiles > INT32_MAX / 2) return cudaErrorInvalidValue;
  const int clusters = (int)std::min<int64_t>(tiles, num_sms() / 2);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * clusters);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // the kernel waits (pdl_wait)
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a0, a1, b0, b1, args, status);
}

int tiles_of(int64_t n, int t) { return (int)((n + t - 1) / t); }

}  // namespace

cudaError_t launch_glu_forward(const void* W_gate, const void* W_up, const void* x, void* h, int64_t N, int D, int H,
                               int act, unsigned* status, cudaStream_t s) {
  if (N <= kGluFewTokens) return launch_glu_few(W_gate, W_up, x, h, (int)N, D, H, act, s);
  CUtensorMap ma, mg, mu;
  if (!make_map_2d(&ma, x, D, N, (uint64_t)D * 2, BK, 128) || !make_map_2d(&mg, W_gate, D, H, (uint64_t)D * 2, BK, 128) ||
      !make_map_2d(&mu, W_up, D, H, (uint64_t)D * 2, BK, 128))
    return cudaErrorInvalidValue;
  GluGemmArgs a{};
  a.M = N;
  a.N = H;
  a.tiles_m = tiles_of(N, 256);
  a.tiles_n = tiles_of(H, 128);
  a.k_blocks = tiles_of(D, BK);
  a.out0 = static_cast<__nv_bfloat16*>(h);
  return act == kActGelu ? launch_mode<GLU_FWD, kActGelu>(ma, ma, mg, mu, a, status, s)
                         : launch_mode<GLU_FWD, kActSilu>(ma, ma, mg, mu, a, status, s);
}

cudaError_t launch_glu_backward(const GluBwdArgs& b, unsigned* status, cudaStream_t s) {
  const int64_t N = b.N;
  const int D = b.D, H = b.H;
  const uint64_t rowD = (uint64_t)D * 2, rowH = (uint64_t)H * 2;
  CUtensorMap a0, a1, b0, b1;
  // dg, du (and h) from x, the weights and dh
  if (!make_map_2d(&a0, b.x, D, N, rowD, BK, 128) || !make_map_2d(&b0, b.W_gate, D, H, rowD, BK, 128) ||
      !make_map_2d(&b1, b.W_up, D, H, rowD, BK, 128))
    return cudaErrorInvalidValue;
  GluGemmArgs g{};
  g.M = N;
  g.N = H;
  g.tiles_m = tiles_of(N, 256);
  g.tiles_n = tiles_of(H, 128);
  g.k_blocks = tiles_of(D, BK);
  g.out0 = static_cast<__nv_bfloat16*>(b.dg);
  g.out1 = static_cast<__nv_bfloat16*>(b.du);
  g.h = static_cast<__nv_bfloat16*>(b.h);
  g.dh = static_cast<const __nv_bfloat16*>(b.dh);
  cudaError_t e = b.act == kActGelu ? launch_mode<GLU_GRAD, kActGelu>(a0, a0, b0, b1, g, status, s)
                                    : launch_mode<GLU_GRAD, kActSilu>(a0, a0, b0, b1, g, status, s);
  if (e != cudaSuccess) return e;
  // dx = dg W_g + du W_u
  if (!make_map_2d(&a0, b.dg, H, N, rowH, BK, 128) || !make_map_2d(&a1, b.du, H, N, rowH, BK, 128) ||
      !make_map_2d(&b0, b.W_gate, D, H, rowD, 64, BK) || !make_map_2d(&b1, b.W_up, D, H, rowD, 64, BK))
    return cudaErrorInvalidValue;
  GluGemmArgs dx{};
  dx.M = N;
  dx.N = D;
  dx.tiles_m = tiles_of(N, 256);
  dx.tiles_n = tiles_of(D, 256);
  dx.kb_half = tiles_of(H, BK);
  dx.k_blocks = 2 * dx.kb_half;
  dx.out0 = static_cast<__nv_bfloat16*>(b.dx);
  e = launch_mode<GLU_DX, kActGelu>(a0, a1, b0, b1, dx, status, s);
  if (e != cudaSuccess) return e;
  // dW_g = dgᵀ x, dW_u = duᵀ x
  if (!make_map_2d(&a0, b.dg, H, N, rowH, 64, BK) || !make_map_2d(&a1, b.du, H, N, rowH, 64, BK) ||
      !make_map_2d(&b0, b.x, D, N, rowD, 64, BK))
    return cudaErrorInvalidValue;
  GluGemmArgs dw{};
  dw.M = H;
  dw.N = D;
  dw.tiles_half = tiles_of(H, 256);
  dw.tiles_m = 2 * dw.tiles_half;
  dw.tiles_n = tiles_of(D, 256);
  dw.k_blocks = tiles_of(N, BK);
  dw.out0 = static_cast<__nv_bfloat16*>(b.dW_gate);
  dw.out1 = static_cast<__nv_bfloat16*>(b.dW_up);
  return launch_mode<GLU_DW, kActGelu>(a0, a1, b0, b0, dw, status, s);
}

}  // namespace rglru
