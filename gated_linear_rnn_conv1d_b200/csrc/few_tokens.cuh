// Products of a few tokens (M ≤ 64) with weight matrices: y = x Wᵀ, or the gated pair
// h = act(x W_gᵀ) ⊙ (x W_uᵀ), forward or with what its backward makes of g and u. Their floor is the weights' way from HBM,
// each byte read once, so the kernel is a stream of weights with the products on the side:
//
// * 16 weight rows are a granule: in the gated form those of 8 channels, the gate's in rows 0–7 and the up
//   projection's in 8–15, so that a thread ends with g and u of the same channel and token. A block has a
//   run of granules, in chunks of up to MT. Its eight warps take the rows' segments (SEG bytes of each row)
//   in turn: a warp forms its segment's products of all the chunk's granules with one load of x.
// * Each warp copies what it needs into a ring of its own in shared memory (cp.async), RING steps of STEP
//   granules' segments, across segment and chunk borders: the bytes in flight that HBM's latency wants cost
//   no registers and no barrier. (TMA boxes of 64 bytes by 16 or 32 rows in the place of these copies were
//   slower: 50 µs against 41 µs for 201 MB of bf16 weights.)
// * Scales of 4-bit weights are brought to shared memory for the block, along the rows: two bytes a row and
//   segment, loaded by the lanes that need them, touched 32 lines a load (12288 gated channels of 4096 inputs,
//   eight tokens, groups of 32: 33 µs, now 19; of 128: 16.2, now 15.2). What is loaded once, x's first
//   segment and the first scales, is asked for before the ring (16.9 µs behind it).
// * The products run on mma.sync m16n8k16 with the weights as the row operand, eight tokens as the
//   columns (the tcgen05 form would want x and unpacked weights in swizzled shared memory for work
//   that is a few percent of the pipe). Lane 4r + t holds row r and r + 8 of the tile. Which k a slot
//   of the MMA stands for is free as long as both operands agree: a lane's slots are neighbouring k.
// * The eight warps' sums meet in shared memory, in a fixed order: results do not depend on the
//   run, nor on how many tokens there are.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

#include "act_math.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace rglru {

constexpr int kFewWarps = 8;
constexpr int kFewThreads = 32 * kFewWarps;

struct FewArgs {
  const uint8_t* w0;             // [rows] rows of row_bytes; the gate's in the gated form
  const uint8_t* w1;             // the up projection's
  const __nv_bfloat16* scales0;  // 4-bit weights: [rows][K / G]
  const __nv_bfloat16* scales1;
  const __nv_bfloat16* x;        // [M][K]
  __nv_bfloat16* out;            // [M][rows], out_ld columns apart
  const __nv_bfloat16* dh;       // the gated form's backward: [M][rows]; out and du are dg and du
  __nv_bfloat16* du;
  __nv_bfloat16* h;              // [M][rows], or null
  int64_t row_bytes;             // a multiple of 16
  int row_groups;                // K / G, or 0
  int M, rows, K, granules, out_ld;
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, bool real) {
  const int bytes = real ? 16 : 0;  // the rest is filled with zeros
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Where byte `byte` of row `row` of a segment lies in shared memory: its 16-byte pieces are permuted within
// the row so that the lanes' reads (READ bytes each: a quad's lanes side by side, eight rows) meet no
// bank twice.
template <int SEG, int READ> __device__ __forceinline__ int seg_offset(int row, int byte) {
  const int f = SEG == 128 ? (READ == 16 ? (row & 1) << 2 : READ == 8 ? (row & 3) << 1 : row & 7)
                           : (READ == 16 ? 0 : READ == 8 ? (row & 2) : (row >> 1) & 3);
  return row * SEG + (((byte / 16) ^ f) * 16) + byte % 16;
}

// bf16 weights.
struct FewBf16 {
  static constexpr int kRead = 16;
  template <int SEG> static constexpr int kGroups = 0;
  static __device__ __forceinline__ int lane_k(int t) { return 8 * t; }
  // x of a segment, as eight-value pieces; the lane's piece c is 32·c further. (x and the scales may be what the kernel
  // ahead writes while this one already lives, which rules the non-coherent loads out.)
  template <int SEG> static constexpr int kX = SEG / 64;
  template <int SEG> static __device__ __forceinline__ uint4 load_x(const FewArgs& a, const __nv_bfloat16* xrow,
                                                                    int seg, int c, int lane) {
    const int k = seg * (SEG / 2) + c * 32;  // beyond K the weights are zeros; x is made so too
    return k + 8 * (lane % 4) < a.K ? *reinterpret_cast<const uint4*>(xrow + k) : make_uint4(0u, 0u, 0u, 0u);
  }
  // x of a segment in the products' order
  template <int NT, int N> static __device__ __forceinline__ void order(uint4 (&)[NT][N]) {}
  // A granule's products with a segment of x.
  template <int NT, int SEG>
  static __device__ __forceinline__ void consume(const uint8_t* smem, const uint32_t*, int, int lane,
                                                 const uint4 (&x)[NT][kX<SEG>], float (&acc)[NT][4]) {
    const int r = lane / 4, t = lane % 4;
#pragma unroll
    for (int c = 0; c < SEG / 64; ++c) {
      const uint4 wa = *reinterpret_cast<const uint4*>(smem + seg_offset<SEG, 16>(r, 64 * c + 16 * t));
      const uint4 wb = *reinterpret_cast<const uint4*>(smem + seg_offset<SEG, 16>(8 + r, 64 * c + 16 * t));
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        mma_bf16(acc[j], wa.x, wb.x, wa.y, wb.y, x[j][c].x, x[j][c].y);
        mma_bf16(acc[j], wa.z, wb.z, wa.w, wb.w, x[j][c].z, x[j][c].w);
      }
    }
  }
};

// 4-bit weights with a bf16 scale for each GROUP inputs of a row: Ŵ = s (q − 8). q − 8 is exact in bf16,
// so a group's sum carries float32's rounding only, and its scale multiplies that sum in float32.
template <int GROUP> struct FewW4 {
  static constexpr int kWords = GROUP / 32;  // of a lane's quarter of a group
  static constexpr int kRead = 4 * kWords;
  template <int SEG> static constexpr int kGroups = 2 * SEG / GROUP;  // of a row's segment
  static __device__ __forceinline__ int lane_k(int t) { return 8 * kWords * t; }
  // Four bf16 pairs (k, k + 4), k = 0 … 3, of a word's eight weights, less 8, by the widely published way of setting an
  // exponent above small integers: 0x4300 is 128, and four bits in the mantissa's last places make 128 + q.
  static __device__ __forceinline__ void unpack(uint32_t w, uint32_t (&p)[4]) {
    const __nv_bfloat162 bias = __floats2bfloat162_rn(136.0f, 136.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t b;  // (w >> 4i) & 0x000F000F | 0x43004300 in one operation after the shift
      asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(b) : "r"(w >> (4 * i)), "r"(0x000F000Fu), "r"(0x43004300u));
      const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&b), bias);
      p[i] = *reinterpret_cast<const uint32_t*>(&d);
    }
  }
  static __device__ __forceinline__ void read(const uint8_t* p, uint32_t (&w)[kWords]) {
    if constexpr (kWords == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if constexpr (kWords == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x; w[1] = v.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
  }
  // x of a segment: piece g·kWords + o is octet o of the lane's quarter of group g
  template <int SEG> static constexpr int kX = 2 * SEG / GROUP * kWords;
  template <int SEG> static __device__ __forceinline__ uint4 load_x(const FewArgs& a, const __nv_bfloat16* xrow,
                                                                    int seg, int c, int) {
    const int k = seg * (2 * SEG) + c / kWords * GROUP;
    return k < a.K ? *reinterpret_cast<const uint4*>(xrow + k + 8 * (c % kWords)) : make_uint4(0u, 0u, 0u, 0u);
  }
  // x of a segment in the unpacked weights' order: pairs (k, k + 4)
  template <int NT, int N> static __device__ __forceinline__ void order(uint4 (&x)[NT][N]) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < N; ++c) {
        const uint4 v = x[j][c];
        x[j][c] = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                             __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
      }
  }
  // A granule's products with a segment of x, which has `groups` groups; scales: of rows r and r + 8.
  template <int NT, int SEG>
  static __device__ __forceinline__ void consume(const uint8_t* smem, const uint32_t* scales, int groups, int lane,
                                                 const uint4 (&x)[NT][kX<SEG>], float (&acc)[NT][4]) {
    const int r = lane / 4, t = lane % 4;
#pragma unroll
    for (int g = 0; g < kGroups<SEG>; ++g) {
      if (g > 0 && g >= groups) break;  // (the same for the whole warp)
      const int byte = g * (GROUP / 2) + t * (4 * kWords);
      const uint32_t f = scales[g];
      uint32_t wa[kWords], wb[kWords];
      read(smem + seg_offset<SEG, kRead>(r, byte), wa);
      read(smem + seg_offset<SEG, kRead>(8 + r, byte), wb);
      float part[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) part[j][c] = 0.0f;
#pragma unroll
      for (int o = 0; o < kWords; ++o) {
        uint32_t da[4], db[4];
        unpack(wa[o], da);
        unpack(wb[o], db);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint4 v = x[j][g * kWords + o];
          mma_bf16(part[j], da[0], db[0], da[1], db[1], v.x, v.y);
          mma_bf16(part[j], da[2], db[2], da[3], db[3], v.z, v.w);
        }
      }
      const float fa = bf16lo(f), fb = bf16hi(f);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        acc[j][0] = fmaf(fa, part[j][0], acc[j][0]);
        acc[j][1] = fmaf(fa, part[j][1], acc[j][1]);
        acc[j][2] = fmaf(fb, part[j][2], acc[j][2]);
        acc[j][3] = fmaf(fb, part[j][3], acc[j][3]);
      }
    }
  }
};

// Scales lie in shared memory in panels of kFewPanel groups of each row, those of rows r and r + 8 of a granule in one
// word.
constexpr int kFewPanel = 64;
constexpr int kFewPanelPitch = kFewPanel + 1;  // words; eight rows' words meet no bank twice

// Shapes of the ring and of the sums: two sum buffers (one barrier a chunk) where they are small.
template <int NT, int MT, int SEG, int STEP, int RING, int GROUPS> struct FewCfg {
  static constexpr int kSegBytes = 16 * STEP * SEG;
  static constexpr int kRingBytes = kFewWarps * RING * kSegBytes;
  static constexpr int kSumFloats = kFewWarps * MT * NT * 4 * 32;
  static constexpr int kSumBufs = MT * NT <= 2 ? 2 : 1;
  static constexpr int kScaleWords = GROUPS > 0 ? 8 * MT * kFewPanelPitch : 0;
  static constexpr int kSmem = kRingBytes + (kSumBufs * kSumFloats + kScaleWords) * 4;
  static constexpr int kBlocks = NT <= 2 || GROUPS == 0 ? 2 : 1;  // per SM (32 tokens' sums and x take 255 registers)
  static_assert(kBlocks * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
};

template <class F, bool GLU, int ACT, int NT, int MT, int SEG, int STEP, int RING, bool GRAD>
__global__ void __launch_bounds__(kFewThreads, FewCfg<NT, MT, SEG, STEP, RING, F::template kGroups<SEG>>::kBlocks)
    few_kernel(FewArgs a) {
  using Cfg = FewCfg<NT, MT, SEG, STEP, RING, F::template kGroups<SEG>>;
  constexpr int kGran = GLU ? 8 : 16;         // output columns of a granule: 16 weight rows
  constexpr int kPieces = SEG / 16;           // of a row's segment
  constexpr int kCopies = 16 * kPieces / 32;  // a lane's copies of a granule's segment
  extern __shared__ __align__(128) uint8_t few_smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  uint8_t* ring = few_smem + warp * RING * Cfg::kSegBytes;
  float* sums = reinterpret_cast<float*>(few_smem + Cfg::kRingBytes);
  const int segs = (int)((a.row_bytes + SEG - 1) / SEG);
  // a block's tokens
  a.x += (int64_t)blockIdx.y * (8 * NT) * a.K;
  a.out += (int64_t)blockIdx.y * (8 * NT) * a.out_ld;
  a.M = min(a.M - (int)blockIdx.y * (8 * NT), 8 * NT);
  const int turns = (segs + kFewWarps - 1) / kFewWarps;
  const int my_segs = segs > warp ? (segs - warp + kFewWarps - 1) / kFewWarps : 0;

  // This block's granules [first, first + count), in chunks of at most MT
  const int each = a.granules / (int)gridDim.x, more = a.granules % (int)gridDim.x;
  const int count = each + ((int)blockIdx.x < more ? 1 : 0);
  const int first = blockIdx.x * each + min((int)blockIdx.x, more);
  const int chunks = (count + MT - 1) / MT;
  const int chunk_each = count / chunks, chunk_more = count % chunks;
  auto chunk_at = [&](int c) { return first + c * chunk_each + min(c, chunk_more); };
  // Before the kernel ahead has ended its results may not be read, but what lies in L2 is the weights whoever
  // wrote them: the first segments are fetched there meanwhile (0.8 µs of 17 or 33).
  {
    constexpr int kLines = kFewWarps * SEG / 128;
    const int n = chunk_at(1) * 16 - first * 16;
    for (int i = threadIdx.x; i < n * kLines; i += kFewThreads) {
      const int row = i / kLines, byte = i % kLines * 128;
      const int at = GLU ? (first + row / 16) * 8 + row % 8 : first * 16 + row;
      const bool up = GLU && row % 16 >= 8;
      const uint8_t* p = (up ? a.w1 : a.w0) + at * a.row_bytes + byte;
      if (at < a.rows && byte < a.row_bytes) asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
      if (F::template kGroups<SEG> > 0 && at < a.rows && byte / 2 < min(a.row_groups, kFewPanel)) {
        const __nv_bfloat16* q = (up ? a.scales1 : a.scales0) + (int64_t)at * a.row_groups + byte / 2;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
      }
    }
  }
  pdl_wait();
  pdl_launch_dependents();

  // The copies' place in the warp's sequence of segments, chunk by chunk. Copy i of a granule takes kStep
  // rows, a lane the piece `piece` of one of them: a block of rows that belongs to one matrix, and that
  // the last granule has whole or not at all (rows is a multiple of 8); rows it has not are computed from
  // what is in shared memory and not stored.
  constexpr int kStep = 32 / kPieces;
  const int piece = lane % kPieces, lr = lane / kPieces;
  int c_chunk = 0, c_left = 0, c_slot = 0, c_m = 0, c_mt = 0, c_rows = 0;
  int64_t c_chunk_at = 0, c_at = 0;  // of this lane's row in the chunk's first granule; and of its piece
  int c_byte = 0;                    // of the row
  const ptrdiff_t up = a.w1 - a.w0;
  auto copy_seg = [&] {
    c_m = 0;
    c_at = c_chunk_at + (c_byte < a.row_bytes ? c_byte : 0);
  };
  auto copy_chunk = [&] {
    const int gr = chunk_at(c_chunk);
    c_mt = chunk_at(c_chunk + 1) - gr;
    c_rows = a.rows - gr * kGran;
    c_chunk_at = (int64_t)(gr * kGran + lr) * a.row_bytes;
    c_byte = warp * SEG + piece * 16;
    c_left = my_segs;
    copy_seg();
  };
  if (my_segs > 0) copy_chunk();
  auto copy_next = [&] {
    if (c_left > 0) {
      const bool real = c_byte < a.row_bytes;
      uint8_t* dst = ring + c_slot * Cfg::kSegBytes;
#pragma unroll
      for (int m = 0; m < STEP; ++m) {
        if (m == 0 || c_m + m < c_mt) {
#pragma unroll
          for (int i = 0; i < kCopies; ++i) {
            const int row = i * kStep;
            const int off = m * kGran + (GLU ? row % 8 : row);
            const uint8_t* src = a.w0 + c_at + off * a.row_bytes + (GLU && row >= 8 ? up : 0);
            if (GLU || c_m * kGran + off < c_rows)
              cp_async_16(smem_u32(dst + seg_offset<SEG, F::kRead>(16 * m + row + lr, 16 * piece)), src, real);
          }
        }
      }
      c_m += STEP;
      c_at += STEP * kGran * a.row_bytes;
      if (c_m >= c_mt) {
        c_byte += kFewWarps * SEG;
        copy_seg();
        if (--c_left == 0 && ++c_chunk < chunks) copy_chunk();
      }
    }
    cp_async_commit();  // (an empty group too: the waits count groups)
    c_slot = c_slot + 1 == RING ? 0 : c_slot + 1;
  };

  // x rows of the lane's tokens (columns beyond M repeat the last token's; they are not stored)
  const __nv_bfloat16* xrow[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
    xrow[j] = a.x + (int64_t)min(8 * j + lane / 4, a.M - 1) * a.K + F::lane_k(lane % 4);
  constexpr int kX = F::template kX<SEG>;
  constexpr bool kEarly = NT * kX <= 4;  // x is loaded a segment ahead (up to 16 registers)
  uint4 x_next[NT][kX];
  auto load_x = [&](uint4(&x)[NT][kX], int seg) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < kX; ++c) x[j][c] = F::template load_x<SEG>(a, xrow[j], seg, c, lane);
  };
  if (kEarly && my_segs > 0) load_x(x_next, warp);

  // A panel's scales of a chunk's rows: warp w takes rows w and w + 8 of each granule, along the rows.
  constexpr int kGroups = F::template kGroups<SEG>;
  constexpr int kPanelSegs = kGroups > 0 ? kFewPanel / (kGroups > 0 ? kGroups : 1) : kFewWarps;
  uint32_t* scales = reinterpret_cast<uint32_t*>(sums + Cfg::kSumBufs * Cfg::kSumFloats);
  struct Scales {
    unsigned short a[MT][kFewPanel / 32], b[MT][kFewPanel / 32];
  };
  auto fetch_scales = [&](Scales& v, int gr, int mt, int panel) {
    const int g0 = panel * kFewPanel + lane;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int n0 = (gr + m) * kGran + warp, n1 = GLU ? n0 : min(n0 + 8, a.rows - 1);
      const unsigned short* s0 = reinterpret_cast<const unsigned short*>(a.scales0) + (int64_t)n0 * a.row_groups + g0;
      const unsigned short* s1 =
          reinterpret_cast<const unsigned short*>(GLU ? a.scales1 : a.scales0) + (int64_t)n1 * a.row_groups + g0;
#pragma unroll
      for (int g = 0; g < kFewPanel / 32; ++g) {
        const bool real = m < mt && g0 + 32 * g < a.row_groups;
        v.a[m][g] = real ? s0[32 * g] : 0;
        v.b[m][g] = real ? s1[32 * g] : 0;
      }
    }
  };
  auto put_scales = [&](const Scales& v, int mt) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int g = 0; g < kFewPanel / 32; ++g)
        if (m < mt)
          scales[(8 * m + warp) * kFewPanelPitch + lane + 32 * g] = (uint32_t)v.a[m][g] | (uint32_t)v.b[m][g] << 16;
  };
  [[maybe_unused]] Scales first_scales;
  if constexpr (kGroups > 0) fetch_scales(first_scales, first, chunk_at(1) - first, 0);
#pragma unroll
  for (int i = 0; i < RING - 1; ++i) copy_next();
  if constexpr (kGroups > 0) put_scales(first_scales, chunk_at(1) - first);

  int slot = 0, buf = 0;
  for (int chunk = 0; chunk < chunks; ++chunk) {
    const int gr = chunk_at(chunk), mt = chunk_at(chunk + 1) - gr;
    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[m][j][c] = 0.0f;
    for (int i = 0; i < turns; ++i) {
      if constexpr (kGroups > 0) {
        constexpr int kPanelTurns = kPanelSegs / kFewWarps;
        if (i % kPanelTurns == 0) {
          if (i > 0 || chunk > 0) {
            if (i > 0) __syncthreads();  // the last panel has been read (the last chunk's: behind its sums' barrier)
            Scales v;
            fetch_scales(v, gr, mt, i / kPanelTurns);
            put_scales(v, mt);
          }
          __syncthreads();
        }
      }
      if (i >= my_segs) break;  // (only in the last turn, past its barriers)
      const int seg = warp + i * kFewWarps;
      uint4 x[NT][kX];
      if (kEarly) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < kX; ++c) x[j][c] = x_next[j][c];
        load_x(x_next, i + 1 == my_segs ? warp : seg + kFewWarps);
      } else {
        load_x(x, seg);
      }
      F::order(x);
      const uint32_t* seg_scales = scales + lane / 4 * kFewPanelPitch + seg % kPanelSegs * kGroups;
      const int groups = a.row_groups - seg * kGroups;
#pragma unroll
      for (int m0 = 0; m0 < MT; m0 += STEP) {
        if (m0 >= mt) break;
        cp_async_wait<RING - 2>();
        __syncwarp();  // the other lanes' pieces too; and all have read the slot that is filled next
        copy_next();
        const uint8_t* smem = ring + slot * Cfg::kSegBytes;
#pragma unroll
        for (int m = 0; m < STEP; ++m)
          if (m0 + m < MT && (m == 0 || m0 + m < mt))
            F::template consume<NT, SEG>(smem + m * 16 * SEG, seg_scales + 8 * (m0 + m) * kFewPanelPitch, groups, lane, x,
                                         acc[m0 + m < MT ? m0 + m : 0]);
        slot = slot + 1 == RING ? 0 : slot + 1;
      }
    }
    float* s = sums + buf * Cfg::kSumFloats;
    if (Cfg::kSumBufs == 1 && chunk > 0) __syncthreads();  // the last chunk's sums have been read
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[((warp * MT + m) * NT * 4 + 4 * j + c) * 32 + lane] = acc[m][j][c];
    // With two buffers: whoever reads this one does so before it comes to the next chunk's barrier,
    // and it is written again after that.
    __syncthreads();
    // A warp adds up one accumulator (two in the gated form) of one granule: element c of token tile j of lane
    // 4r + t is row r + 8·(c / 2) of token 8j + 2t + c % 2.
    constexpr int kElems = GLU ? 2 : 4;
    for (int i = warp; i < mt * NT * kElems; i += kFewWarps) {
      const int c = i % kElems, j = i / kElems % NT, m = i / (kElems * NT);
      const float* p = s + (m * NT * 4 + 4 * j + c) * 32 + lane;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) v += p[w * MT * NT * 4 * 32];
      const int token = 8 * j + 2 * (lane % 4) + c % 2, col = (gr + m) * kGran + 8 * (c / 2) + lane / 4;
      [[maybe_unused]] float u = 0.0f, slope;
      if constexpr (GLU) {
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) u += p[w * MT * NT * 4 * 32 + 64];
      }
      if (token >= a.M || col >= a.rows) continue;
      const int64_t at = (int64_t)token * a.out_ld + col;
      if constexpr (GRAD) {  // (roundings as the tiles': glu.cu)
        const float d = __bfloat162float(a.dh[(int64_t)token * a.rows + col]), act = v * act_gate<ACT, true>(v, slope);
        a.out[at] = __float2bfloat16_rn(d * u * slope);
        a.du[at] = __float2bfloat16_rn(d * act);
        if (a.h != nullptr) a.h[(int64_t)token * a.rows + col] = __float2bfloat16_rn(act * u);
      } else {
        if constexpr (GLU) v = v * act_gate<ACT, false>(v, slope) * u;
        a.out[at] = __float2bfloat16_rn(v);
      }
    }
    if (Cfg::kSumBufs == 2) buf ^= 1;
  }
  cp_async_wait<0>();
}

template <class F, bool GLU, int ACT, int NT, int MT, int SEG, int STEP, int RING, bool GRAD = false>
cudaError_t launch_few(FewArgs a, cudaStream_t s) {
  using Cfg = FewCfg<NT, MT, SEG, STEP, RING, F::template kGroups<SEG>>;
  auto kern = few_kernel<F, GLU, ACT, NT, MT, SEG, STEP, RING, GRAD>;
  static bool attr_set[64] = {};  // idempotent: a race sets it twice
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  a.granules = (a.rows + (GLU ? 7 : 15)) / (GLU ? 8 : 16);
  const int y = (a.M + 8 * NT - 1) / (8 * NT);
  const int room = num_sms() * Cfg::kBlocks / y;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.granules < room ? a.granules : room, y);
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = Cfg::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // the kernel waits (pdl_wait)
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace rglru
