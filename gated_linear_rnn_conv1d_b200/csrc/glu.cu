// The gated feed-forward block ("Griffin：将门控线性循环与局部注意力混合以实现高效的语言模型",
// §MLP块 (gated MLP, Fig. 2(b))) without its down projection, and its backward:
//     g = x W_gᵀ,  u = x W_uᵀ,  h = act(g) ⊙ u,              x [N][D], W_g, W_u [H][D]
//     dg = dh ⊙ u ⊙ act'(g),  du = dh ⊙ act(g)               (g and u formed again from x)
//     dx = dg W_g + du W_u,   dW_g = dgᵀ x,  dW_u = duᵀ x.
// The forward is two products of 2·N·D·H operations each, the backward six (g, u, two for dx, one for each dW). With many
// tokens the tensor cores bound every part, so the elementwise work rides in the products' epilogues and g, u are never
// stored.
//
// One kernel shape: persistent CTA pairs (cta_group::2) on output tiles of up to 256 × 256, as the gate
// GEMM's: warp 0 loads by TMA, warp 1 of the leader issues the MMAs, eight warps of each CTA
// empty one accumulator while the next tile's MMAs fill the other. Three modes of it:
//   GLU_FWD   h: rank 0 stages 128 rows of W_g, rank 1 the same 128 rows of W_u, so a tile holds
//             g in columns 0–127 and u of the same channels in 128–255.
//   GLU_GRAD  the same products; the epilogue reads dh and writes dg, du (and h when asked for).
//             (Up to kGluFewTokens tokens glu_few.cu does what these two do.)
//   GLU_WIDE  dx, dW_g and dW_u in one launch: [dg | du]·[W_g; W_u] with the weights read in place as
//             an MN-major operand, k over dg's channels and then over du's; dgᵀx and duᵀx with both
//             operands MN-major in place, k over the tokens.
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
constexpr int kMaxStages = 16;
constexpr int kABytes = 128 * BK * 2;  // this CTA's 128 rows of A
constexpr int kBBytes = 128 * BK * 2;  // this CTA's half of the B tile
// The ring has as many stages as fit, of the rows that are loaded (set_ring): the bytes in flight are what HBM's
// latency asks for. Of weights that are not in L2, D 4096, H 12288, 64 tokens take 51.3 µs and 57.3 with six
// stages of the largest; 256 tokens 57.3 and 61.3; from 2048 tokens on there is no difference. An MMA reads 128
// rows of A whatever was loaded: up to kABytes from a k-block's start have to be there.
constexpr int kRingBytes = 7 * (kABytes + kBBytes);
constexpr int kSmem = kRingBytes + 1024;
// Tiles of dW whose k is short leave by TMA, from two boxes of 32 rows × 64 columns for each epilogue warp, behind a
// smaller ring.
constexpr int kBoxBytes = 32 * 64 * 2, kBoxes = 2;
constexpr int kTmemCols = 512;  // two 256-column accumulators
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kAllBoxes = kEpiWarps * kBoxes * kBoxBytes;
// Output tiles are taken in bands of kBand tile rows, column by column: the 74 pairs at work at
// a time then cover about 8 × 9 tiles, whose operands (17 · 256 rows of k) stay in L2 between them.
constexpr int kBand = 8;

enum GluMode { GLU_FWD = 0, GLU_GRAD = 1, GLU_WIDE = 2 };

// A product's output: tiles_m × tiles_n tiles of 2·half_rows rows (each CTA's half, up to 128; where there
// are few tokens, no more than they need: the MMA's other rows are made of what shared memory holds
// and not stored) and `width` columns.
struct GluProduct {
  int64_t M;             // output rows
  int tiles_m, half_rows;
  int k_blocks;
  // a stage of the ring: `group` k-blocks of kb_bytes each, B's rows b_at from a k-block's start
  int group, b_at, kb_bytes;
  __nv_bfloat16* out;
  // k may be cut into `splits` pieces of kb_per k-blocks, each a tile of its own that writes its float32 sums
  // to part [splits][M][N]; a second kernel adds them, in order
  int splits, kb_per;
  float* part;
};

struct GluGemmArgs {
  int N;               // output columns: H channels (GLU_FWD, GLU_GRAD) or D
  int stages, stage_bytes;  // the ring
  int staged, least;        // dW leaves through shared memory; what a tile costs at least (tile_cost)
  int tiles_n, width;  // of every product; width: channels (up to 128), or columns (up to 256)
  int ld;              // columns between the rows of out and du (GLU_GRAD: of the scratch dg and du)
  int wide, wide_h;    // rows of out and du, of h, start on 32-byte borders
  __nv_bfloat16* du;          // GLU_GRAD
  __nv_bfloat16* h;           // GLU_GRAD: h, or null
  const __nv_bfloat16* dh;    // GLU_GRAD
  int kb_half;         // dx: k-blocks of dg (du's follow)
  // p[0]: h or dg; or dx. p[1], p[2]: dW_g and dW_u, whose tiles are numbered through.
  GluProduct p[3];
  // How the tiles are dealt out. First the tiles with the longer k (dx's, or with dw_first dW's), one to
  // each pair in turn; the pairs that the last turn leaves out (all but the first `rest`) take
  // `extra` short ones in their place; the other short ones go round again, those pairs first.
  int dw_first, n_long, n_short, rest, extra;
};

struct Tile {
  int m, n, which, split, kb0, kb1;
};
// The it-th tile of a pair; false when it has no more.
template <int MODE>
__device__ __forceinline__ bool tile_of(const GluGemmArgs& a, int it, int pair, int pairs, Tile& t) {
  int64_t at = (int64_t)it * pairs + pair;
  bool is_long = true;
  if (at >= a.n_long) {
    if (MODE != GLU_WIDE) return false;
    is_long = false;
    const bool late = pair >= a.rest;  // left out of the last turn
    int i = it - (a.n_long - pair + pairs - 1) / pairs;
    const int others = pairs - a.rest;
    if (late && i < a.extra) {
      at = (int64_t)i * others + pair - a.rest;
    } else {
      if (late) i -= a.extra;
      at = (int64_t)a.extra * others + (int64_t)i * pairs + (late ? pair - a.rest : pair + others);
    }
    if (at >= a.n_short) return false;
  }
  int tile = (int)at;
  t.which = 0;
  if (MODE == GLU_WIDE && is_long == (a.dw_first != 0)) {  // a tile of dW
    const int each = a.p[1].tiles_m * a.tiles_n * a.p[1].splits;
    t.which = tile < each ? 1 : 2;
    tile -= tile < each ? 0 : each;
  }
  const int tiles_m = t.which == 0 ? a.p[0].tiles_m : a.p[1].tiles_m;
  t.split = 0;
  t.kb0 = 0;
  t.kb1 = t.which == 0 ? a.p[0].k_blocks : a.p[1].k_blocks;
  if constexpr (MODE == GLU_WIDE) {
    const int kb_per = t.which == 0 ? a.p[0].kb_per : a.p[1].kb_per;
    t.split = tile / (tiles_m * a.tiles_n);
    tile -= t.split * tiles_m * a.tiles_n;
    t.kb0 = t.split * kb_per;
    t.kb1 = min(t.kb0 + kb_per, t.kb1);
  }
  const int band = tile / (kBand * a.tiles_n);
  const int r = tile - band * kBand * a.tiles_n;
  const int rows = min(kBand, tiles_m - band * kBand);
  t.n = r / rows;
  t.m = band * kBand + r - t.n * rows;
  return true;
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// Sixteen columns of a row, from column `col` of `cols`: one 32-byte store where the rows allow it (a whole
// sector of L2; two 16-byte stores are written as three), else one for each eight columns that exist.
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&v)[16], int col, int cols, int wide) {
  const uint4 a = pack8(v), b = pack8(v + 8);
  if (wide && col + 16 <= cols) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    if (col < cols) *reinterpret_cast<uint4*>(p) = a;
    if (col + 8 < cols) *reinterpret_cast<uint4*>(p + 8) = b;
  }
}

// The same for rows that may start in the middle of a sector (ODD kernels): such a row's second eight columns wait for
// the next sixteen, so that its sectors too are stored whole, but for the first and the last (forward of 26090 tokens,
// D 208, H 8952: 434 µs with stores of 16 bytes, 336 so; backward of one token, D 2072, H 5224: 45.7 and 40.3).
struct RowStore {
  uint4 held;
  bool odd;
  __device__ __forceinline__ explicit RowStore(const void* row)
      : held(make_uint4(0u, 0u, 0u, 0u)), odd((reinterpret_cast<uintptr_t>(row) & 16u) != 0) {}
  // columns col … col + 15; `first`: of the thread's
  __device__ __forceinline__ void put(__nv_bfloat16* p, const float (&v)[16], int col, int cols, bool first) {
    if (!odd) {
      store16(p, v, col, cols, 1);
      return;
    }
    const uint4 a = pack8(v), b = pack8(v + 8);
    if (col >= cols) {
      if (!first) flush(p, col, cols);
    } else if (first) {
      *reinterpret_cast<uint4*>(p) = a;
    } else {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p - 8), "r"(held.x), "r"(held.y),
                   "r"(held.z), "r"(held.w), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w)
                   : "memory");
    }
    held = b;
  }
  // after the last: p, col are the next column's
  __device__ __forceinline__ void flush(__nv_bfloat16* p, int col, int cols) const {
    if (odd && col - 8 < cols) *reinterpret_cast<uint4*>(p - 8) = held;
  }
};

// (part's rows are multiples of 32 bytes, as D is of eight)
__device__ __forceinline__ void store8_f32(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// As mbar_wait, the thread asleep between its looks (the epilogue's and the loader's waits are long;
// looking all the time costs issue slots and power).
__device__ __forceinline__ bool wait_asleep(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait_sleep(a, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (mbar_try_wait_sleep(a, parity)) return true;
    if (*abort || clock64() - t0 > kWaitCycles) return false;
  }
}

// GROUP: 1 where every stage has one k-block. STAGED: dW's tiles leave through shared memory by TMA.
// ODD: rows of out that may start off a sector's border
template <int MODE, int ACT, int GROUP, bool STAGED, bool ODD>
__global__ void __launch_bounds__(kThreads, 1)
    glu_gemm_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1,
                    const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1,
                    const __grid_constant__ CUtensorMap tmC0, const __grid_constant__ CUtensorMap tmC1,
                    const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmO1,
                    const __grid_constant__ CUtensorMap tmO2, const GluGemmArgs args, unsigned* status) {
  // GLU_FWD, GLU_GRAD: A0 x, B0 W_g, B1 W_u. GLU_WIDE: A0 dg, A1 du, B0 W_g, B1 W_u (for dx); C0 dg, C1 du,
  // X x (for dW, in boxes of 64 columns).
  constexpr bool kGated = MODE != GLU_WIDE;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[kMaxStages];
  __shared__ __align__(8) uint64_t empty_bar[kMaxStages];
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

  if (threadIdx.x == 0) {
    for (int i = 0; i < args.stages; ++i) {
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
    tma_prefetch_desc(&tmB1);
    if (!kGated) {
      tma_prefetch_desc(&tmA1);
      tma_prefetch_desc(&tmC0);
      tma_prefetch_desc(&tmC1);
      tma_prefetch_desc(&tmX);
      if (STAGED) {
        tma_prefetch_desc(&tmO1);
        tma_prefetch_desc(&tmO2);
      }
    }
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
    // The whole warp runs the loop and one lane issues: addresses and coordinates then stay in uniform
    // registers, where TMA and MMA instructions take them from. A loop of one lane alone moves each of them
    // over, which cost the MMA warp 572 cycles a k-block whatever the tile's width; now it is 525 for the
    // widest tile (512 of them the MMAs') and 397 for three quarters of it.
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    // this CTA's half of the tile's columns: `width` weight rows, or in one or two boxes of 64 columns
    const int half_cols = kGated ? args.width : args.width / 2;
    const bool two = !kGated && half_cols > 64;
    const uint32_t b_bytes = kGated ? half_cols * BK * 2 : two ? kBBytes : kBBytes / 2;
    Tile t;
    for (int it = 0; ok && tile_of<MODE>(args, it, cluster, n_clusters, t); ++it) {
      const int half_rows = t.which == 0 ? args.p[0].half_rows : 128;
      const int arow = (2 * t.m + (int)rank) * half_rows;
      const uint32_t bytes = 2 * (half_rows * BK * 2 + b_bytes);
      const GluProduct& p = kGated || t.which == 0 ? args.p[0] : args.p[1];
      const int group = GROUP == 1 ? 1 : p.group, b_at = p.b_at, kb_bytes = p.kb_bytes;
      const int bcol = kGated ? t.n * args.width : t.n * args.width + (int)rank * half_cols;
      const bool is_dx = kGated || t.which == 0;
      const bool second = !kGated && t.which == 2;
      for (int kb = t.kb0; kb < t.kb1; kb += group) {
        ok = __all_sync(0xffffffffu, wait_asleep(&empty_bar[stage], phase ^ 1, &abort_s));
        if (!ok) break;
        uint8_t* stage_at = smem + stage * args.stage_bytes;
        const uint32_t lbar = leader_full0 + stage * 8;
        const int n = GROUP == 1 ? 1 : min(group, t.kb1 - kb);
        const uint32_t stage_tx = n * bytes;
        auto load = [&](int k, uint8_t* sa) {  // (by one lane)
          uint8_t* sb = sa + b_at;
          if constexpr (kGated) {
            tma_load_2d_2sm(sa, &tmA0, lbar, k * BK, arow);
            tma_load_2d_2sm(sb, leader ? &tmB0 : &tmB1, lbar, k * BK, bcol);
          } else {
            // an MN-major operand: 128 columns as two boxes of 64 columns × BK rows
            const bool du = k >= args.kb_half;
            const int kc = (is_dx && du ? k - args.kb_half : k) * BK;
            const CUtensorMap* mb = is_dx ? (du ? &tmB1 : &tmB0) : &tmX;
            if (is_dx) {
              tma_load_2d_2sm(sa, du ? &tmA1 : &tmA0, lbar, kc, arow);
            } else {
              tma_load_2d_2sm(sa, second ? &tmC1 : &tmC0, lbar, arow, kc);
              tma_load_2d_2sm(sa + kABytes / 2, second ? &tmC1 : &tmC0, lbar, arow + 64, kc);
            }
            tma_load_2d_2sm(sb, mb, lbar, bcol, kc);
            if (two) tma_load_2d_2sm(sb + kBBytes / 2, mb, lbar, bcol + 64, kc);
          }
        };
        if (elect_one()) {
          if (leader) mbar_arrive_expect_tx(&full_bar[stage], stage_tx);
          load(kb, stage_at);
          if constexpr (GROUP > 1)
            for (int i = 1; i < n; ++i) load(kb + i, stage_at + i * kb_bytes);
        }
        __syncwarp();
        if (++stage == args.stages) { stage = 0; phase ^= 1; }
      }
    }
    // What is under way to this CTA's shared memory arrives before the CTA may end: the last MMAs' arrivals on its
    // empty barriers; and after a wait that ran out the copies themselves, which the leader's full barriers count for
    // both CTAs.
    for (int i = 0; ok && i < args.stages; ++i)
      ok = __all_sync(0xffffffffu, wait_asleep(&empty_bar[i], i < stage ? phase : phase ^ 1, &abort_s));
    if (!ok) {
      if (lane == 0) { abort_s = 1; atomicOr(status, kStatusTimeout); }
      volatile int never = 0;
      bool there = leader;
      for (int i = 0; there && i < args.stages; ++i)
        there = __all_sync(0xffffffffu, mbar_wait(&full_bar[i], i < stage ? phase : phase ^ 1, &never));
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (leader CTA only) ----------------
    if (leader) {
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      const uint32_t idesc = umma_idesc_bf16_f32(256, kGated ? 2 * args.width : args.width);
      const uint32_t smem0 = smem_u32(smem);
      Tile t;
      for (int it = 0; ok && tile_of<MODE>(args, it, cluster, n_clusters, t); ++it) {
        const bool a_mn = !kGated && t.which != 0;
        ok = __all_sync(0xffffffffu, mbar_wait(&tempty_bar[acc], acc_phase ^ 1, &abort_s));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * 256;
        const GluProduct& p = kGated || t.which == 0 ? args.p[0] : args.p[1];
        const int group = GROUP == 1 ? 1 : p.group, b_at = p.b_at, kb_bytes = p.kb_bytes;
        for (int kb = t.kb0; kb < t.kb1; kb += group) {
          ok = __all_sync(0xffffffffu, mbar_wait(&full_bar[stage], phase, &abort_s));
          if (!ok) break;
          tc_fence_after();
          const uint32_t stage_at = smem0 + stage * args.stage_bytes;
          const uint32_t first = kb == t.kb0 ? 0u : 1u;
          // one MMA takes 16 of k: 32 bytes along K-major rows, 16 rows of 128 B of an MN-major box (in
          // units of 16 bytes, the descriptors' start address)
          struct Block {
            uint64_t a_k, b_k, a_m, b_m;
          };
          auto block = [&](uint32_t a_addr) {
            const uint32_t b_addr = a_addr + b_at;
            return Block{umma_desc_sw128(a_addr), umma_desc_sw128(b_addr), umma_desc_sw128_mn(a_addr, kABytes / 2),
                         umma_desc_sw128_mn(b_addr, kBBytes / 2)};
          };
          auto issue = [&](const Block& d, uint32_t first) {  // (by one lane)
            if (kGated) {
#pragma unroll
              for (int k = 0; k < BK / 16; ++k)
                umma_f16_2sm(d_tmem, d.a_k + k * 2, d.b_k + k * 2, idesc, k == 0 ? first : 1u);
            } else if (a_mn) {
#pragma unroll
              for (int k = 0; k < BK / 16; ++k)
                umma_f16_2sm(d_tmem, d.a_m + k * 128, d.b_m + k * 128, idesc | kIdescAMN | kIdescBMN, k == 0 ? first : 1u);
            } else {
#pragma unroll
              for (int k = 0; k < BK / 16; ++k)
                umma_f16_2sm(d_tmem, d.a_k + k * 2, d.b_m + k * 128, idesc | kIdescBMN, k == 0 ? first : 1u);
            }
          };
          const Block b0 = block(stage_at);
          if (elect_one()) {
            issue(b0, first);
            if constexpr (GROUP > 1)
              for (int i = 1; i < min(group, t.kb1 - kb); ++i) issue(block(stage_at + i * kb_bytes), 1u);
            umma_commit_2sm_both(&empty_bar[stage]);
          }
          __syncwarp();
          if (++stage == args.stages) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
        if (elect_one()) umma_commit_2sm_both(&tfull_bar[acc]);
        __syncwarp();
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
      if (!ok && lane == 0) { abort_s = 1; atomicOr(status, kStatusTimeout); }
      // every MMA issued here has completed before TMEM is freed
      if (elect_one())
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                         smem_u32(&drain_bar))
                     : "memory");
      __syncwarp();
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
    // the pairs of 16 columns this warp takes: half of the width's
    const int pieces = args.width / (kGated ? 16 : 32);
    const int first = half * ((pieces + 1) / 2), count = half == 0 ? (pieces + 1) / 2 : pieces / 2;
    constexpr int kStep = kGated ? 16 : 32;
    [[maybe_unused]] int box_at = 0;  // STAGED: the box in use
    [[maybe_unused]] uint8_t* const boxes = smem + kRingBytes - kAllBoxes + (warp - 2) * kBoxes * kBoxBytes;
    Tile t;
    for (int it = 0; tile_of<MODE>(args, it, cluster, n_clusters, t); ++it) {
      const int64_t rows = kGated || t.which == 0 ? args.p[0].M : args.p[1].M;
      __nv_bfloat16* out = kGated || t.which == 0 ? args.p[0].out : t.which == 1 ? args.p[1].out : args.p[2].out;
      const int half_rows = t.which == 0 ? args.p[0].half_rows : 128;
      const int64_t row = (int64_t)(2 * t.m + rank) * half_rows + quarter * 32 + lane;
      const bool row_ok = row < rows && quarter * 32 + lane < half_rows;
      const int col0 = t.n * args.width + first * kStep;
      const int64_t base = row * args.ld + col0;
      // dh of this thread's row, loaded before the accumulator is ready (coherently: it may be what the kernel ahead wrote
      // while this one already lived)
      [[maybe_unused]] uint4 dhq[MODE == GLU_GRAD ? 8 : 1];
      if constexpr (MODE == GLU_GRAD) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          dhq[q] = row_ok && q < 2 * count && col0 + 8 * q < args.N
                       ? reinterpret_cast<const uint4*>(args.dh + row * args.N + col0)[q]
                       : make_uint4(0u, 0u, 0u, 0u);
      }
      if (!wait_asleep(&tfull_bar[acc], acc_phase, &abort_s)) {
        abort_s = 1;
        atomicOr(status, kStatusTimeout);
        break;
      }
      tc_fence_after();
      const uint32_t t_row = tmem_base + ((uint32_t)(quarter * 32) << 16) + acc * 256;
      [[maybe_unused]] RowStore odd_row(out + base);
      // four pairs of 16 columns; the next pair's TMEM loads are in flight while one is worked on
      const uint32_t ta = t_row + first * kStep, tb = ta + (kGated ? args.width : 16);
      uint32_t ra[2][16], rb[2][16];
      tmem_ld_x16(ta, ra[0]);
      tmem_ld_x16(tb, rb[0]);
      tmem_ld_wait16(ra[0], rb[0]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k >= count) break;
        const int cur = k & 1;
        if (k + 1 < count) {
          tmem_ld_x16(ta + (k + 1) * kStep, ra[cur ^ 1]);
          tmem_ld_x16(tb + (k + 1) * kStep, rb[cur ^ 1]);
        }
        const int col = col0 + k * kStep;
        const int64_t at = base + k * kStep;
        float o0[16], o1[16];
        if constexpr (kGated) {
          [[maybe_unused]] float o2[16];
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            const float2 g = make_float2(__uint_as_float(ra[cur][j]), __uint_as_float(ra[cur][j + 1]));
            const float2 u = make_float2(__uint_as_float(rb[cur][j]), __uint_as_float(rb[cur][j + 1]));
            float2 slope;
            const float2 a = __fmul2_rn(g, act_gate2<ACT, MODE == GLU_GRAD>(g, slope));
            const float2 hv = __fmul2_rn(a, u);
            if constexpr (MODE == GLU_FWD) {
              o0[j] = hv.x;
              o0[j + 1] = hv.y;
            } else {
              const uint4 d4 = dhq[2 * k + j / 8];
              const uint32_t w = j % 8 == 0 ? d4.x : j % 8 == 2 ? d4.y : j % 8 == 4 ? d4.z : d4.w;
              const float2 d = make_float2(bf16lo(w), bf16hi(w));
              // dg and du are rounded to bf16, the operands of the next products: half a step of 2^-8
              // each, as much as the rounding of dx and dW themselves
              const float2 dg = __fmul2_rn(__fmul2_rn(d, u), slope), du = __fmul2_rn(d, a);
              o0[j] = dg.x;
              o0[j + 1] = dg.y;
              o1[j] = du.x;
              o1[j + 1] = du.y;
              o2[j] = hv.x;
              o2[j + 1] = hv.y;
            }
          }
          if (row_ok) {
            if constexpr (ODD)
              odd_row.put(out + at, o0, col, args.N, k == 0);
            else
              store16(out + at, o0, col, args.N, args.wide);
            if constexpr (MODE == GLU_GRAD) {
              store16(args.du + at, o1, col, args.N, args.wide);
              if (args.h != nullptr) store16(args.h + row * args.N + col, o2, col, args.N, args.wide_h);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            o0[j] = __uint_as_float(ra[cur][j]);
            o1[j] = __uint_as_float(rb[cur][j]);
          }
          float* part = t.which == 0 ? args.p[0].part : t.which == 1 ? args.p[1].part : args.p[2].part;
          if (STAGED && t.which != 0) {
            // a piece is half of a box: 64 of a row's 128 bytes, in 16-byte chunks permuted as the tensor map's
            // swizzle has them (eight rows' chunks meet no bank twice)
            uint8_t* box = boxes + box_at * kBoxBytes;
            if ((k & 1) == 0) {
              if (lane == 0) bulk_wait_read<kBoxes - 1>();  // the box's last store has been read (the others' may not)
              __syncwarp();
            }
            const uint4 q[4] = {pack8(o0), pack8(o0 + 8), pack8(o1), pack8(o1 + 8)};
#pragma unroll
            for (int c = 0; c < 4; ++c)
              *reinterpret_cast<uint4*>(box + lane * 128 + (((k & 1) * 4 + c) ^ (lane & 7)) * 16) = q[c];
            if ((k & 1) == 1) {
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                const int r0 = (2 * t.m + (int)rank) * 128 + quarter * 32, c0 = col - 32;
                if (r0 < rows && c0 < args.N) tma_store_2d(t.which == 1 ? &tmO1 : &tmO2, box, c0, r0);
                bulk_commit();
              }
              box_at = box_at + 1 == kBoxes ? 0 : box_at + 1;
            }
          } else if (row_ok && part == nullptr) {
            if constexpr (ODD) {
              odd_row.put(out + at, o0, col, args.N, k == 0);
              odd_row.put(out + at + 16, o1, col + 16, args.N, false);
            } else {
              store16(out + at, o0, col, args.N, args.wide);
              store16(out + at + 16, o1, col + 16, args.N, args.wide);
            }
          } else if (row_ok) {
            part += (int64_t)t.split * rows * args.N + at;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              if (col + 8 * q < args.N) store8_f32(part + 8 * q, &o0[8 * q]);
              if (col + 16 + 8 * q < args.N) store8_f32(part + 16 + 8 * q, &o1[8 * q]);
            }
          }
        }
        if (k + 1 < count) tmem_ld_wait16(ra[cur ^ 1], rb[cur ^ 1]);
      }
      if constexpr (ODD) {
        const float* part = kGated || t.which == 0 ? args.p[0].part : args.p[1].part;
        if (row_ok && count > 0 && part == nullptr)
          odd_row.flush(out + base + count * kStep, col0 + count * kStep, args.N);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(leader_tempty0 + acc * 8);
      if (++acc == 2) { acc = 0; acc_phase ^= 1; }
    }
    if (STAGED && lane == 0) bulk_wait();
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

// out = Σ part[s] for up to three outputs: eight values a thread, splits added in order.
struct GluSum {
  const float* part;
  __nv_bfloat16* out;
  int64_t n8;  // vectors of eight
  int splits;
};
struct GluSums {
  GluSum s[3];
};
__global__ void __launch_bounds__(256) glu_sum_kernel(const GluSums a) {
  pdl_wait();
  pdl_launch_dependents();
  int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const GluSum& u = a.s[k];
    if (i >= 0 && i < u.n8) {
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      const float4* p = reinterpret_cast<const float4*>(u.part) + 2 * i;
#pragma unroll 4
      for (int s = 0; s < u.splits; ++s) {
        const float4 x = __ldcs(p + 2 * u.n8 * s), y = __ldcs(p + 2 * u.n8 * s + 1);
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
      }
      reinterpret_cast<uint4*>(u.out)[i] = pack8(v);
    }
    i -= u.n8;
  }
}

struct Maps {
  CUtensorMap a0, a1, b0, b1, c0, c1, x, o1, o2;
};

template <int MODE, int ACT, int GROUP, bool STAGED = false, bool ODD = false>
cudaError_t launch_group(const Maps& m, const GluGemmArgs& args, int pairs, unsigned* status, cudaStream_t s) {
  auto kern = glu_gemm_kernel<MODE, ACT, GROUP, STAGED, ODD>;
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
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
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
  return cudaLaunchKernelEx(&cfg, kern, m.a0, m.a1, m.b0, m.b1, m.c0, m.c1, m.x, m.o1, m.o2, args, status);
}

template <int MODE, int ACT>
cudaError_t launch_mode(const Maps& m, const GluGemmArgs& args, int pairs, unsigned* status, cudaStream_t s) {
  const bool one = args.p[0].group == 1 && (MODE != GLU_WIDE || args.p[1].group == 1);
  if constexpr (MODE == GLU_WIDE) {
    if (args.staged)
      return one ? launch_group<MODE, ACT, 1, true>(m, args, pairs, status, s)
                 : launch_group<MODE, ACT, 2, true>(m, args, pairs, status, s);
  }
  if constexpr (MODE != GLU_GRAD) {
    if (!args.wide)
      return one ? launch_group<MODE, ACT, 1, false, true>(m, args, pairs, status, s)
                 : launch_group<MODE, ACT, 2, false, true>(m, args, pairs, status, s);
  }
  return one ? launch_group<MODE, ACT, 1>(m, args, pairs, status, s) : launch_group<MODE, ACT, 2>(m, args, pairs, status, s);
}

int tiles_of(int64_t n, int t) { return (int)((n + t - 1) / t); }
bool on32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

// What a tile of so many k-blocks costs in k-blocks (of about 0.3 µs): its accumulator changes hands, and
// where its k is short the epilogue is what it takes: twelve for 256 × 256 of dW stored by the threads, each a row of
// its own, eight where they leave by TMA (D 4096, H 12288: 16 tokens 153 → 139 µs, 64 tokens 157 → 144, 256 tokens
// 172 → 162; D 2048, H 6144: 44.8 → 40.0, 48.0 → 43.9, 55.3 → 51.6; the shortest of several runs, their middle is up to
// 15 % longer).
int tile_cost(int k_blocks, int least) { return std::max(k_blocks + 2, least); }

// The ring. A product's k-block has half_rows of A and b_bytes of B (multiples of 1024 bytes). Handing a stage over
// costs the issuing warp 0.12 µs and its MMAs 0.10 µs a k-block for 32 channels (0.14 for 64, 0.28 for 128): with
// narrow tiles a stage has up to four k-blocks, as long as five stages fit (four of dx's and dW's). D 4096, H 2048:
// 64 tokens 29 → 16.7 µs, 256 tokens 18.5 → 14.6; D 256, H 768, 64 tokens backward 13.2 → 9.9. Tiles of 128 channels
// keep one: their MMAs hide the handing over, and the loop over a stage's k-blocks, which one lane runs, costs
// them 4 % (hence two kernels).
void set_ring(GluGemmArgs& g, int products, int b_bytes, int ring) {
  int reach = 0;  // an MMA reads kABytes from a k-block's start whatever was loaded
  int most = products == 1 ? (ring - kABytes) / 5 : ring / 4;
  g.stage_bytes = 0;
  for (int i = products - 1; i >= 0; --i) {
    GluProduct& p = g.p[i];
    p.b_at = p.half_rows * BK * 2;
    p.kb_bytes = p.b_at + b_bytes;
    p.group = std::max(1, std::min(4, most / p.kb_bytes));
    g.stage_bytes = std::max(g.stage_bytes, p.group * p.kb_bytes);
    most = g.stage_bytes;  // (dx's k-blocks fit dW's stages)
    reach = std::max(reach, (p.group - 1) * p.kb_bytes + std::max(kABytes, p.kb_bytes));
  }
  g.stages = std::min(kMaxStages, (ring - std::max(0, reach - g.stage_bytes)) / g.stage_bytes);
}

// Deals out n_long tiles of `a` k-blocks and n_short of `b` ≤ a to `pairs` CTA pairs (GluGemmArgs); returns the
// longest share.
int64_t deal(int64_t n_long, int a, int64_t n_short, int b, int pairs, GluGemmArgs& g) {
  g.n_long = (int)n_long;
  g.n_short = (int)n_short;
  g.rest = (int)(n_long % pairs);
  const int others = pairs - g.rest;
  a = tile_cost(a, g.least);
  b = tile_cost(b, g.least);
  g.extra = g.rest == 0 || n_short == 0 ? 0 : (int)std::min<int64_t>(a / b, n_short / others);
  const int64_t turns = n_long / pairs, left = n_short - (int64_t)g.extra * others;
  const int64_t again = left / pairs, more = left % pairs;
  const int64_t late = turns * a + (g.extra + again + (more > 0 ? 1 : 0)) * (int64_t)b;
  const int64_t early = (turns + 1) * a + (again + (more > others ? 1 : 0)) * (int64_t)b;
  return g.rest == 0 ? late : std::max(late, early);
}

// The tile width in steps of `step` up to `most` with the shortest longest share, a k-block's cost
// being what it loads, half_rows of A and half the width's rows of B for each CTA. (A width that leaves few
// columns over and fills the last turn; at equal cost the wider.)
template <class F> int best_width(int cols, int most, int step, int half_rows, F share) {
  int best = most;
  double least = 0;
  for (int w = most; w >= std::max(step, most / 4); w -= step) {
    const double c = share(tiles_of(cols, w)) * (half_rows / 128.0 + (double)w / most);
    if (w == most || c < 0.97 * least) {
      best = w;
      least = c;
    }
  }
  return best;
}

GluProduct product(int64_t rows, int k_blocks, void* out) {
  const int tiles = tiles_of(rows, 256);
  GluProduct p{};
  p.M = rows;
  p.tiles_m = tiles;
  p.half_rows = 8 * tiles_of(rows, 16 * tiles);
  p.k_blocks = p.kb_per = k_blocks;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.splits = 1;
  return p;
}

// dx, dW_g and dW_u: the tile width, and in how many pieces of k they are formed. A product whose k-blocks are
// many more than a pair's share of all the work (few tokens and a long H for dx; many tokens and small
// weights for dW) is cut into pieces of about that share, at least 16 k-blocks long; the second kernel
// and the partial sums cost about as much as 16 more. A function of the sizes alone (74 pairs, a B200's),
// as the workspace holds the partial sums.
constexpr int kPairs = 74;
int64_t share_wide(GluGemmArgs& w, int tiles_n, int pairs) {
  const int64_t n_dx = (int64_t)w.p[0].tiles_m * tiles_n * w.p[0].splits;
  const int64_t n_dw = 2 * (int64_t)w.p[1].tiles_m * tiles_n * w.p[1].splits;
  w.dw_first = w.p[1].kb_per > w.p[0].kb_per;
  return w.dw_first ? deal(n_dw, w.p[1].kb_per, n_dx, w.p[0].kb_per, pairs, w)
                    : deal(n_dx, w.p[0].kb_per, n_dw, w.p[1].kb_per, pairs, w);
}
int64_t cut_wide(GluGemmArgs& w, int tiles_n) {
  const int64_t n_dx = (int64_t)w.p[0].tiles_m * tiles_n, n_dw = 2 * (int64_t)w.p[1].tiles_m * tiles_n;
  const int64_t all = n_dx * tile_cost(w.p[0].k_blocks, w.least) + n_dw * tile_cost(w.p[1].k_blocks, w.least);
  const int64_t share = std::max<int64_t>(all / kPairs, 16);
  int64_t more = 0;
  for (int i = 0; i < 3; ++i) {
    GluProduct& p = w.p[i];
    p.splits = 1;
    p.kb_per = p.k_blocks;
    if (4 * (int64_t)p.k_blocks > 5 * share && p.k_blocks >= share + 16) {
      p.splits = tiles_of(p.k_blocks, (int)share);
      p.kb_per = tiles_of(p.k_blocks, p.splits);
      p.splits = tiles_of(p.k_blocks, p.kb_per);
      more = 16;
    }
  }
  return share_wide(w, tiles_n, kPairs) + more;
}
void plan_wide(int64_t N, int D, int H, GluGemmArgs& w) {
  w = GluGemmArgs{};
  w.N = w.ld = D;
  w.kb_half = tiles_of(H, BK);
  w.p[0] = product(N, 2 * w.kb_half, nullptr);
  w.p[1] = product(H, tiles_of(N, BK), nullptr);
  w.p[1].half_rows = 128;  // (read in boxes of 64 columns)
  w.p[2] = w.p[1];
  // (below a tile a pair there is nothing to gain, D 256, H 768, 16 tokens 8.4 µs and staged 9.7; nor where rows are no
  // whole lines, D 1032, H 2888, 100 tokens 25.0 and 26.9; nor from 512 tokens on, D 2048, H 6144 71.2 and 71.6)
  w.staged = w.p[1].k_blocks <= 6 && D % 64 == 0 && 2 * w.p[1].tiles_m * tiles_of(D, 256) >= kPairs;
  w.least = w.staged ? 8 : 12;
  w.width = best_width(D, 256, w.staged ? 128 : 32, 128, [&](int tiles_n) { return (double)cut_wide(w, tiles_n); });
  w.tiles_n = tiles_of(D, w.width);
  set_ring(w, 3, w.width > 128 ? kBBytes : kBBytes / 2, kRingBytes - (w.staged ? kAllBoxes : 0));
  cut_wide(w, w.tiles_n);
}
int64_t part_floats(const GluProduct& p, int D) { return p.splits > 1 ? p.splits * p.M * D : 0; }

// g and u of N tokens: the tensor maps and the tiles of GLU_FWD and GLU_GRAD.
bool gated_args(const void* W_gate, const void* W_up, const void* x, void* out, int64_t N, int D, int H, Maps& m,
                GluGemmArgs& a, int& pairs) {
  a = GluGemmArgs{};
  a.N = a.ld = H;
  a.least = 12;
  a.p[0] = product(N, tiles_of(D, BK), out);
  const int room = num_sms() / 2;
  a.width = best_width(H, 128, 16, a.p[0].half_rows, [&](int tiles_n) {
    return (double)deal((int64_t)a.p[0].tiles_m * tiles_n, a.p[0].k_blocks, 0, 0, room, a);
  });
  a.tiles_n = tiles_of(H, a.width);
  set_ring(a, 1, a.width * BK * 2, kRingBytes);
  const int64_t tiles = (int64_t)a.p[0].tiles_m * a.tiles_n;
  if (tiles > INT32_MAX / 2) return false;
  pairs = (int)std::min<int64_t>(tiles, room);
  deal(tiles, a.p[0].k_blocks, 0, 0, pairs, a);
  const uint64_t row = (uint64_t)D * 2;
  if (!make_map_2d(&m.a0, x, D, N, row, BK, a.p[0].half_rows) || !make_map_2d(&m.b0, W_gate, D, H, row, BK, a.width) ||
      !make_map_2d(&m.b1, W_up, D, H, row, BK, a.width))
    return false;
  m.a1 = m.c0 = m.c1 = m.x = m.o1 = m.o2 = m.a0;  // (not read)
  return true;
}

}  // namespace

cudaError_t launch_glu_forward(const void* W_gate, const void* W_up, const void* x, void* h, int64_t N, int D, int H,
                               int act, unsigned* status, cudaStream_t s) {
  if (N <= kGluFewTokens) return launch_glu_few(W_gate, W_up, x, h, (int)N, D, H, act, s);
  Maps m;
  GluGemmArgs a;
  int pairs;
  if (!gated_args(W_gate, W_up, x, h, N, D, H, m, a, pairs)) return cudaErrorInvalidValue;
  a.wide = H % 16 == 0 && on32(h);
  return act == kActGelu ? launch_mode<GLU_FWD, kActGelu>(m, a, pairs, status, s)
                         : launch_mode<GLU_FWD, kActSilu>(m, a, pairs, status, s);
}

cudaError_t launch_glu_backward(const GluBwdArgs& b, unsigned* status, cudaStream_t s) {
  const int64_t N = b.N;
  const int D = b.D, H = b.H;
  // dg, du (and h) from x, the weights and dh
  Maps m{};
  int pairs;
  cudaError_t e;
  if (N <= kGluFewTokens) {
    e = launch_glu_few_grad(b, s);
  } else {
    GluGemmArgs a;
    if (!gated_args(b.W_gate, b.W_up, b.x, b.dg, N, D, H, m, a, pairs)) return cudaErrorInvalidValue;
    a.du = static_cast<__nv_bfloat16*>(b.du);
    a.h = static_cast<__nv_bfloat16*>(b.h);
    a.dh = static_cast<const __nv_bfloat16*>(b.dh);
    a.ld = glu_scratch_pitch(H);
    a.wide = on32(b.dg) && on32(b.du);
    a.wide_h = H % 16 == 0 && on32(b.h);
    e = b.act == kActGelu ? launch_mode<GLU_GRAD, kActGelu>(m, a, pairs, status, s)
                          : launch_mode<GLU_GRAD, kActSilu>(m, a, pairs, status, s);
  }
  if (e != cudaSuccess) return e;
  // dx = dg W_g + du W_u, dW_g = dgᵀ x, dW_u = duᵀ x
  const uint64_t rowD = (uint64_t)D * 2, rowH = (uint64_t)glu_scratch_pitch(H) * 2;
  GluGemmArgs w;
  plan_wide(N, D, H, w);
  w.wide = D % 16 == 0 && on32(b.dx) && on32(b.dW_gate) && on32(b.dW_up);
  void* const outs[3] = {b.dx, b.dW_gate, b.dW_up};
  float* part = static_cast<float*>(b.part);
  GluSums sums{};
  int64_t vectors = 0;
  for (int i = 0; i < 3; ++i) {
    w.p[i].out = static_cast<__nv_bfloat16*>(outs[i]);
    if (w.p[i].splits == 1) continue;
    w.p[i].part = part;
    sums.s[i] = GluSum{part, w.p[i].out, w.p[i].M * D / 8, w.p[i].splits};
    part += part_floats(w.p[i], D);
    vectors += sums.s[i].n8;
  }
  if (!make_map_2d(&m.a0, b.dg, H, N, rowH, BK, w.p[0].half_rows) ||
      !make_map_2d(&m.a1, b.du, H, N, rowH, BK, w.p[0].half_rows) ||
      !make_map_2d(&m.b0, b.W_gate, D, H, rowD, 64, BK) || !make_map_2d(&m.b1, b.W_up, D, H, rowD, 64, BK) ||
      !make_map_2d(&m.c0, b.dg, H, N, rowH, 64, BK) || !make_map_2d(&m.c1, b.du, H, N, rowH, 64, BK) ||
      !make_map_2d(&m.x, b.x, D, N, rowD, 64, BK))
    return cudaErrorInvalidValue;
  if (w.staged && (!make_map_2d(&m.o1, b.dW_gate, D, H, rowD, 64, 32) || !make_map_2d(&m.o2, b.dW_up, D, H, rowD, 64, 32)))
    return cudaErrorInvalidValue;
  const int64_t tiles = ((int64_t)w.p[0].tiles_m * w.p[0].splits + 2 * (int64_t)w.p[1].tiles_m * w.p[1].splits) * w.tiles_n;
  if (tiles > INT32_MAX / 2 || (vectors + 255) / 256 > INT32_MAX) return cudaErrorInvalidValue;
  pairs = (int)std::min<int64_t>(tiles, num_sms() / 2);
  share_wide(w, w.tiles_n, pairs);
  e = launch_mode<GLU_WIDE, kActGelu>(m, w, pairs, status, s);
  if (e != cudaSuccess || vectors == 0) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((vectors + 255) / 256));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // the kernel waits (pdl_wait)
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, glu_sum_kernel, (const GluSums)sums);
}

size_t glu_backward_part_bytes(int64_t N, int D, int H) {
  GluGemmArgs w;
  plan_wide(N, D, H, w);
  return (size_t)(part_floats(w.p[0], D) + part_floats(w.p[1], D) + part_floats(w.p[2], D)) * sizeof(float);
}

}  // namespace rglru
