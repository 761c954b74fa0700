// Activation checkpoints in 8 bits: x [rows][C] as int8 codes and one power of two for each group
// of 32 channels (the last group of a row may be short). For a group with largest magnitude m,
//     e = the smallest integer ≥ −127 with |rint(x / 2^e)| ≤ 127,   code = rint(x / 2^e),   x̂ = code · 2^e,
// stored as e + 127 (0 … 249), or 255 for a group that holds an infinity or a NaN, which comes back
// as NaN. Scaling by a power of two is exact and a code has seven bits, so the one rounding is
// rint's: |x̂ − x| ≤ 2^(e−1), at most 1/127 of m, and x̂ is a bfloat16 number: the tensor cores take
// it as it is. Both kernels are bound by HBM: 2 (4) bytes of x and 33/32 of the checkpoint a channel.
#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>

#include "kernels.cuh"
#include "ptx.cuh"

namespace rglru {
namespace {

constexpr int kThreads8 = 256;
constexpr int kGroup = kAct8Group;
constexpr uint32_t kInfBits = 0x7F800000u;

// Where item i is: an item is eight channels, four neighbouring lanes hold a group. kWhole: C is a
// multiple of 32, so items are numbered through; otherwise rows are padded to whole groups
// (vp items, v8 of them real).
struct Item {
  int64_t vec;    // index among vectors of eight channels
  int64_t group;  // index among groups
  bool real;
};
template <bool kWhole> __device__ __forceinline__ Item item_of(int64_t i, int vp, int v8) {
  if constexpr (kWhole) return {i, i >> 2, true};
  const int64_t row = i / vp;
  const int v = (int)(i - row * vp);
  return {row * v8 + v, i >> 2, v < v8};
}

template <typename T> struct Vec8;
template <> struct Vec8<__nv_bfloat16> {
  uint4 q;
  __device__ void load(const void* p, int64_t vec) { q = __ldcs(static_cast<const uint4*>(p) + vec); }
  __device__ void get(float (&f)[8]) const {
    f[0] = bf16lo(q.x); f[1] = bf16hi(q.x); f[2] = bf16lo(q.y); f[3] = bf16hi(q.y);
    f[4] = bf16lo(q.z); f[5] = bf16hi(q.z); f[6] = bf16lo(q.w); f[7] = bf16hi(q.w);
  }
  static __device__ void store(void* p, int64_t vec, const float (&f)[8]) {
    static_cast<uint4*>(p)[vec] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                             pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
};
template <> struct Vec8<float> {
  float4 a, b;
  __device__ void load(const void* p, int64_t vec) {
    a = __ldcs(static_cast<const float4*>(p) + 2 * vec);
    b = __ldcs(static_cast<const float4*>(p) + 2 * vec + 1);
  }
  __device__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  static __device__ void store(void* p, int64_t vec, const float (&f)[8]) {
    static_cast<float4*>(p)[2 * vec] = make_float4(f[0], f[1], f[2], f[3]);
    static_cast<float4*>(p)[2 * vec + 1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

template <typename T, bool kWhole>
__global__ void __launch_bounds__(kThreads8)
    act8_pack_kernel(const void* __restrict__ x, uint2* __restrict__ codes, uint8_t* __restrict__ scales,
                     int64_t items, int vp, int v8) {
  // items is a multiple of 4, so a group's four lanes are all inside or all outside
  const int64_t i = (int64_t)blockIdx.x * kThreads8 + threadIdx.x;
  const bool in = i < items;
  const Item it = item_of<kWhole>(in ? i : 0, vp, v8);
  Vec8<T> v;
  float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (in && it.real) {
    v.load(x, it.vec);
    v.get(f);
  }
  uint32_t top = 0;  // magnitudes compare as their bits do; infinities and NaN are above the rest
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(f[j]) & 0x7FFFFFFFu);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  // e + 127: m / 2^e is in [64, 128) for e = ⌊log₂ m⌋ − 6, and one more is needed from 127.5 on,
  // which rint takes to 128
  int e = (int)(top >> 23) - 6;
  if (e >= 0 && __uint_as_float(top) * __uint_as_float((uint32_t)(254 - e) << 23) >= 127.5f) ++e;
  e = max(e, 0);
  const bool finite = top < kInfBits;
  const float inv = finite ? __uint_as_float((uint32_t)(254 - e) << 23) : 0.0f;
  if (!in) return;
  if ((threadIdx.x & 3) == 0) scales[it.group] = finite ? (uint8_t)e : (uint8_t)255;
  if (!it.real) return;
  uint32_t w[2] = {0u, 0u};
  if (finite) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j / 4] |= (uint32_t)(__float2int_rn(f[j] * inv) & 0xFF) << (8 * (j % 4));
  }
  codes[it.vec] = make_uint2(w[0], w[1]);
}

template <typename T, bool kWhole>
__global__ void __launch_bounds__(kThreads8)
    act8_unpack_kernel(const uint2* __restrict__ codes, const uint8_t* __restrict__ scales, void* __restrict__ x,
                       int64_t items, int vp, int v8) {
  const int64_t i = (int64_t)blockIdx.x * kThreads8 + threadIdx.x;
  if (i >= items) return;
  const Item it = item_of<kWhole>(i, vp, v8);
  if (!it.real) return;
  const uint2 w = __ldcs(codes + it.vec);
  const uint32_t e = scales[it.group];
  // 2^(e − 127): e = 0 is subnormal
  const float step = e == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(e > 0u ? e << 23 : 1u << 22);
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = (float)(int8_t)((j < 4 ? w.x : w.y) >> (8 * (j % 4))) * step;
  Vec8<T>::store(x, it.vec, f);
}

}  // namespace

cudaError_t launch_act8_pack(const void* x, void* codes, void* scales, int64_t rows, int C, bool bf16,
                             cudaStream_t s) {
  const bool whole = C % kGroup == 0;
  const int v8 = C / 8, vp = (C + kGroup - 1) / kGroup * 4;
  const int64_t items = rows * vp;
  const int64_t blocks = (items + kThreads8 - 1) / kThreads8;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  auto kern = bf16 ? (whole ? act8_pack_kernel<__nv_bfloat16, true> : act8_pack_kernel<__nv_bfloat16, false>)
                   : (whole ? act8_pack_kernel<float, true> : act8_pack_kernel<float, false>);
  kern<<<(unsigned)blocks, kThreads8, 0, s>>>(x, static_cast<uint2*>(codes), static_cast<uint8_t*>(scales), items, vp,
                                              v8);
  return cudaGetLastError();
}

cudaError_t launch_act8_unpack(const void* codes, const void* scales, void* x, int64_t rows, int C, bool bf16,
                               cudaStream_t s) {
  const bool whole = C % kGroup == 0;
  const int v8 = C / 8, vp = (C + kGroup - 1) / kGroup * 4;
  const int64_t items = rows * vp;
  const int64_t blocks = (items + kThreads8 - 1) / kThreads8;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  auto kern = bf16 ? (whole ? act8_unpack_kernel<__nv_bfloat16, true> : act8_unpack_kernel<__nv_bfloat16, false>)
                   : (whole ? act8_unpack_kernel<float, true> : act8_unpack_kernel<float, false>);
  kern<<<(unsigned)blocks, kThreads8, 0, s>>>(static_cast<const uint2*>(codes), static_cast<const uint8_t*>(scales),
                                              x, items, vp, v8);
  return cudaGetLastError();
}

}  // namespace rglru
