// Products of a few tokens with 4-bit weights, for serving: y = x Ŵᵀ and the gated pair
// h = act(x Ŵ_gᵀ) ⊙ (x Ŵ_uᵀ), x [M][K] bf16 with M ≤ 64,
//     Ŵ[n][k] = s[n][k / G] · (q[n][k] − 8),   q in 4 bits (even k in the low half of a byte), s bf16.
// HBM bounds them: half a byte a weight and 2 / G of scale. The products themselves run on the
// tensor cores (mma.sync m16n8k16: a warp's weights go from HBM through registers, where they are
// unpacked, straight into the A operand; tcgen05 would want them unpacked in shared memory
// first, as much traffic there as the unpacking itself): q − 8 is a small integer, exact in
// bf16, so a group's sum carries no rounding but float32's, and its scale multiplies that sum in
// float32, once for each of 16 rows × 8 tokens.
//
// A block takes 16 weight rows (or 8 channels: rows 0–7 of the tile are the gate's, 8–15 the up
// projection's, so a thread ends with both of the same channel and token); its eight warps take
// the groups in turn and their sums meet in shared memory, in a fixed order. Lane 4r + t reads
// G/8 bytes (G/4 weights) of rows r and r + 8: a quad's four pieces are one group. Which k an
// MMA's slot stands for is free as long as both operands agree: slots are filled in the order that
// unpacks cheapest, a word's k and k + 4 side by side.
#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>

#include "act_math.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace rglru {
namespace {

constexpr int kW4Warps = 8;
constexpr int kW4Threads = 32 * kW4Warps;

struct W4Args {
  const uint8_t* codes0;  // [rows][K / 2]
  const __nv_bfloat16* scales0;  // [rows][K / G]
  const uint8_t* codes1;  // the up projection's
  const __nv_bfloat16* scales1;
  const __nv_bfloat16* x;  // [M][K]
  __nv_bfloat16* out;      // [M][rows]
  int M, rows, K;
};

// Four bf16 pairs (k, k + 4), k = 0 … 3, of a word's eight weights, less 8: 0x4300 is 128, and a
// number of four bits in the mantissa's last place makes 128 + q.
__device__ __forceinline__ void unpack_w4(uint32_t w, uint32_t (&p)[4]) {
  const __nv_bfloat162 bias = __floats2bfloat162_rn(136.0f, 136.0f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&b), bias);
    p[i] = *reinterpret_cast<const uint32_t*>(&d);
  }
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Words of a lane's piece of a group: G / 32.
template <int WORDS> __device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[WORDS]) {
  if constexpr (WORDS == 4) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else if constexpr (WORDS == 2) {
    const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
    w[0] = v.x; w[1] = v.y;
  } else {
    w[0] = __ldcs(reinterpret_cast<const uint32_t*>(p));
  }
}

// GLU: two weights, eight channels a block. NT: tiles of eight tokens.
template <int GROUP, bool GLU, int ACT, int NT>
__global__ void __launch_bounds__(kW4Threads)
    w4_kernel(const W4Args a) {
  constexpr int WORDS = GROUP / 32;
  __shared__ float sums[kW4Warps][NT * 4][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int r = lane / 4, t = lane % 4;
  constexpr int kRows = GLU ? 8 : 16;
  const int row0 = blockIdx.x * kRows;
  const int groups = a.K / GROUP;
  // this lane's two weight rows (a linear's last tile may have eight rows; the others are
  // computed from the last row again and not stored)
  const int rowA = row0 + r, rowB = GLU ? rowA : min(rowA + 8, a.rows - 1);
  const uint8_t* pA = a.codes0 + (int64_t)rowA * (a.K / 2) + t * (4 * WORDS);
  const uint8_t* pB = (GLU ? a.codes1 : a.codes0) + (int64_t)rowB * (a.K / 2) + t * (4 * WORDS);
  const __nv_bfloat16* sA = a.scales0 + (int64_t)rowA * groups;
  const __nv_bfloat16* sB = (GLU ? a.scales1 : a.scales0) + (int64_t)rowB * groups;

  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[j][c] = 0.0f;

#pragma unroll 2
  for (int g = warp; g < groups; g += kW4Warps) {
    uint32_t wa[WORDS], wb[WORDS];
    load_words<WORDS>(pA + (int64_t)g * (GROUP / 2), wa);
    load_words<WORDS>(pB + (int64_t)g * (GROUP / 2), wb);
    const float fa = __bfloat162float(sA[g]), fb = __bfloat162float(sB[g]);
    float part[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) part[j][c] = 0.0f;
#pragma unroll
    for (int o = 0; o < WORDS; ++o) {
      uint32_t da[4], db[4];
      unpack_w4(wa[o], da);
      unpack_w4(wb[o], db);
      const int k = g * GROUP + t * (8 * WORDS) + 8 * o;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int token = 8 * j + r;
        uint4 xv = make_uint4(0u, 0u, 0u, 0u);
        if (token < a.M) xv = __ldg(reinterpret_cast<const uint4*>(a.x + (int64_t)token * a.K + k));
        mma_bf16(part[j], da[0], db[0], da[1], db[1], __byte_perm(xv.x, xv.z, 0x5410), __byte_perm(xv.x, xv.z, 0x7632));
        mma_bf16(part[j], da[2], db[2], da[3], db[3], __byte_perm(xv.y, xv.w, 0x5410), __byte_perm(xv.y, xv.w, 0x7632));
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      acc[j][0] = fmaf(fa, part[j][0], acc[j][0]);
      acc[j][1] = fmaf(fa, part[j][1], acc[j][1]);
      acc[j][2] = fmaf(fb, part[j][2], acc[j][2]);
      acc[j][3] = fmaf(fb, part[j][3], acc[j][3]);
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int c = 0; c < 4; ++c) sums[warp][4 * j + c][lane] = acc[j][c];
  __syncthreads();
  // outputs, rows fastest: value (row, token) of the tile is element (token & 1) + 2·(row / 8) of
  // lane 4·(row & 7) + (token & 7) / 2
  for (int i = threadIdx.x; i < kRows * 8 * NT; i += kW4Threads) {
    const int row = i % kRows, token = i / kRows;
    const int at = 4 * (token / 8) + (token & 1), ln = 4 * (row & 7) + (token & 7) / 2;
    if (token >= a.M || row0 + row >= a.rows) continue;
    float v = 0.0f, u = 0.0f;
    if constexpr (GLU) {
#pragma unroll
      for (int w = 0; w < kW4Warps; ++w) {
        v += sums[w][at][ln];
        u += sums[w][at + 2][ln];
      }
      float none;
      v = v * act_gate<ACT, false>(v, none) * u;
    } else {
#pragma unroll
      for (int w = 0; w < kW4Warps; ++w) v += sums[w][at + 2 * (row / 8)][ln];
    }
    a.out[(int64_t)token * a.rows + row0 + row] = __float2bfloat16_rn(v);
  }
}

template <int GROUP, bool GLU, int ACT> cudaError_t launch_group(const W4Args& a, cudaStream_t s) {
  const int rows = GLU ? 8 : 16;
  const int blocks = (a.rows + rows - 1) / rows;
  auto kern = a.M <= 8    ? w4_kernel<GROUP, GLU, ACT, 1>
              : a.M <= 16 ? w4_kernel<GROUP, GLU, ACT, 2>
              : a.M <= 32 ? w4_kernel<GROUP, GLU, ACT, 4>
                          : w4_kernel<GROUP, GLU, ACT, 8>;
  kern<<<blocks, kW4Threads, 0, s>>>(a);
  return cudaGetLastError();
}

template <bool GLU, int ACT> cudaError_t launch_any(const W4Args& a, int group, cudaStream_t s) {
  switch (group) {
    case 32: return launch_group<32, GLU, ACT>(a, s);
    case 64: return launch_group<64, GLU, ACT>(a, s);
    case 128: return launch_group<128, GLU, ACT>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

// Quantisation: a thread forms one group of one row. s = bf16(max |w| / 7), q = rint(w / s) + 8, the
// divisions IEEE float32's; |w / s| ≤ 7·(1 + 2^-8), so q stays in 1 … 15 wherever s is a normal
// number (below, it is held there). A group of zeros gets s = 0 and q = 8; one that holds an
// infinity or a NaN gets s = NaN.
template <int GROUP>
__global__ void __launch_bounds__(128)
    w4_quantize_kernel(const __nv_bfloat16* __restrict__ w, uint8_t* __restrict__ codes,
                       __nv_bfloat16* __restrict__ scales, int64_t n_groups) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n_groups) return;
  const uint4* src = reinterpret_cast<const uint4*>(w + i * GROUP);
  uint4 v[GROUP / 8];
  uint32_t top = 0;  // magnitudes compare as their bits do; infinities and NaN are above the rest
#pragma unroll
  for (int j = 0; j < GROUP / 8; ++j) {
    v[j] = __ldg(src + j);
    const uint32_t q[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) top = max(top, max((q[k] << 16) & 0x7FFF0000u, q[k] & 0x7FFF0000u));
  }
  const __nv_bfloat16 sb = __float2bfloat16_rn(
      top < 0x7F800000u ? __fdiv_rn(__uint_as_float(top), 7.0f) : __uint_as_float(0x7FC00000u));
  const float s = __bfloat162float(sb);
  scales[i] = sb;
  uint32_t* dst = reinterpret_cast<uint32_t*>(codes + i * (GROUP / 2));
#pragma unroll
  for (int j = 0; j < GROUP / 8; ++j) {
    const uint32_t q[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
    uint32_t word = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float f = k % 2 == 0 ? bf16lo(q[k / 2]) : bf16hi(q[k / 2]);
      const int c = s > 0.0f ? min(max(__float2int_rn(__fdiv_rn(f, s)), -7), 7) + 8 : 8;
      word |= (uint32_t)c << (4 * k);
    }
    dst[j] = word;
  }
}

}  // namespace

cudaError_t launch_w4_quantize(const void* w, void* codes, void* scales, int64_t rows, int K, int group,
                               cudaStream_t s) {
  const int64_t n = rows * (K / group);
  const int64_t blocks = (n + 127) / 128;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  auto kern = group == 32 ? w4_quantize_kernel<32> : group == 64 ? w4_quantize_kernel<64> : w4_quantize_kernel<128>;
  kern<<<(unsigned)blocks, 128, 0, s>>>(static_cast<const __nv_bfloat16*>(w), static_cast<uint8_t*>(codes),
                                        static_cast<__nv_bfloat16*>(scales), n);
  return cudaGetLastError();
}

cudaError_t launch_w4_linear(const W4Matrix& w, const void* x, void* y, int M, int rows, int K, int group,
                             cudaStream_t s) {
  W4Args a{};
  a.codes0 = static_cast<const uint8_t*>(w.codes);
  a.scales0 = static_cast<const __nv_bfloat16*>(w.scales);
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.out = static_cast<__nv_bfloat16*>(y);
  a.M = M;
  a.rows = rows;
  a.K = K;
  return launch_any<false, kActGelu>(a, group, s);
}

cudaError_t launch_w4_glu(const W4Matrix& gate, const W4Matrix& up, const void* x, void* h, int M, int rows, int K,
                          int group, int act, cudaStream_t s) {
  W4Args a{};
  a.codes0 = static_cast<const uint8_t*>(gate.codes);
  a.scales0 = static_cast<const __nv_bfloat16*>(gate.scales);
  a.codes1 = static_cast<const uint8_t*>(up.codes);
  a.scales1 = static_cast<const __nv_bfloat16*>(up.scales);
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.out = static_cast<__nv_bfloat16*>(h);
  a.M = M;
  a.rows = rows;
  a.K = K;
  return act == kActGelu ? launch_any<true, kActGelu>(a, group, s) : launch_any<true, kActSilu>(a, group, s);
}

}  // namespace rglru
