// Activation checkpoints in 8 bits: x [rows][C] as int8 codes and one power of two for each group
// of 32 channels (the last group of a row may be short). For a group with largest magnitude m,
//     e = the smallest integer ≥ −127 with |rint(x / 2^e)| ≤ 127,   code = rint(x / 2^e),   x̂ = code · 2^e,
// stored as e + 127 (0 … 248), or 255 for a group that holds an infinity or a NaN, which comes back
// as NaN. Scaling by a power of two is exact and a code has seven bits, so the one rounding is
// rint's: |x̂ − x| ≤ 2^(e−1), at most 1/127 of m, and x̂ is a bfloat16 number: the tensor cores take
// it as it is. From m = 127.5·2^121 on e would be 122 and m itself 64·2^122 = 2^128, which is no finite number: there e
// stays 121 and codes are held within ±127, which is off by less than 2^121, at most 1/127 of m as well.
// Both kernels are bound by HBM: 2 (4) bytes of x and 33/32 of the checkpoint a channel.
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
constexpr int kTopScale = 121 + 127;

// Where item i is: an item is eight channels, four neighbouring lanes hold a group. kWhole: C is a
// multiple of 32, so items are numbered through; otherwise rows are padded to whole groups
// (vp items, v8 of them real).
struct Item {
  int64_t vec;    // index among vectors of eight channels
  int64_t group;  // index among groups
  bool real;
};
// Groups n < 2^30 over the groups of a row, d, without a division: ⌊n / d⌋ = ⌊n·mul / 2^shift⌋ for mul = ⌈2^shift / d⌉ and
// 2^shift ≥ 2^30·d (mul·d exceeds 2^shift by less than d ≤ 2^(shift − 30): Granlund and Montgomery, "Division by
// invariant integers using multiplication", 1994). 4096 × 4104 bf16: pack 11.4 µs, unpack 7.8, and 12.3 and 9.3 with
// divisions of 32 bits; 16384 rows 42.5 and 34.1, and 45.0 and 35.9 (C = 4096: 34.1 and 33.6).
struct RowOf {
  uint32_t mul;
  int shift;
};
RowOf row_of(int d) {
  int shift = 30;
  while ((1 << (shift - 30)) < d) ++shift;
  return {(uint32_t)((((uint64_t)1 << shift) + d - 1) / d), shift};
}
// A thread's items, a block's width apart: the u-th is item `at`.
template <bool kWhole> struct Walk {
  int64_t row = 0;
  int v = 0;
  __device__ __forceinline__ Item next(int u, int64_t at, int64_t items, int vp, int v8, RowOf d) {
    if constexpr (kWhole) {
      return {at, at >> 2, at < items};
    } else {
      if (u == 0 || vp < kThreads8) {
        row = at < (int64_t)1 << 32 ? (int64_t)(((uint64_t)((uint32_t)at >> 2) * d.mul) >> d.shift) : at / vp;
        v = (int)(at - row * vp);
      } else if ((v += kThreads8) >= vp) {  // (rows at least as long as a block: at most one further)
        v -= vp;
        ++row;
      }
      return {at - row * (vp - v8), at >> 2, v < v8 && at < items};
    }
  }
};

template <typename T> struct Vec8;
template <> struct Vec8<__nv_bfloat16> {
  uint4 q;
  __device__ void load(const void* p, int64_t vec) { q = __ldcs(static_cast<const uint4*>(p) + vec); }
  __device__ void get(float (&f)[8]) const {
    f[0] = bf16lo(q.x); f[1] = bf16hi(q.x); f[2] = bf16lo(q.y); f[3] = bf16hi(q.y);
    f[4] = bf16lo(q.z); f[5] = bf16hi(q.z); f[6] = bf16lo(q.w); f[7] = bf16hi(q.w);
  }
  // magnitudes held within 127·2^121, whose bits are 0x7F7E (on the packed values, in the rare branch that needs it, the
  // pack kernel keeps its time: 130.8 µs both ways, 133.5 with the eight floats held, 139.5 without the branch)
  __device__ void hold() {
    const uint32_t lim = 0x7F7E7F7Eu;
    auto h = [&](uint32_t a) { return (a & 0x80008000u) | __vminu2(a & 0x7FFF7FFFu, lim); };
    q.x = h(q.x); q.y = h(q.y); q.z = h(q.z); q.w = h(q.w);
  }
  // the bits of the largest magnitude, as a float32's
  __device__ uint32_t top() const {
    const uint32_t m = __vmaxu2(__vmaxu2(q.x & 0x7FFF7FFFu, q.y & 0x7FFF7FFFu),
                                __vmaxu2(q.z & 0x7FFF7FFFu, q.w & 0x7FFF7FFFu));
    return max(m & 0xFFFF0000u, m << 16);
  }
  static __device__ void store(void* p, int64_t vec, const float (&f)[8], bool) {
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
  __device__ void hold() {
    auto h = [](float x) { return fminf(fmaxf(x, -127.0f * 0x1p121f), 127.0f * 0x1p121f); };
    a = make_float4(h(a.x), h(a.y), h(a.z), h(a.w));
    b = make_float4(h(b.x), h(b.y), h(b.z), h(b.w));
  }
  __device__ uint32_t top() const {
    uint32_t m = 0;
    const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7FFFFFFFu);
    return m;
  }
  // wide: p is on a 32-byte border, and the eight values make one store of a whole L2 sector
  static __device__ void store(void* p, int64_t vec, const float (&f)[8], bool wide) {
    float* d = static_cast<float*>(p) + 8 * vec;
    if (wide) {
      asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(d), "f"(f[0]), "f"(f[1]), "f"(f[2]),
                   "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                   : "memory");
    } else {
      reinterpret_cast<float4*>(d)[0] = make_float4(f[0], f[1], f[2], f[3]);
      reinterpret_cast<float4*>(d)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
  }
};

// A thread takes kItems items, a block's width apart, and loads them all before it works on the first.
template <typename T> constexpr int kItems = sizeof(T) == 2 ? 4 : 2;

template <typename T, bool kWhole>
__global__ void __launch_bounds__(kThreads8)
    act8_pack_kernel(const void* __restrict__ x, uint2* __restrict__ codes, uint8_t* __restrict__ scales,
                     int64_t items, int vp, int v8, RowOf row) {
  constexpr int U = kItems<T>;
  // items is a multiple of 4, so a group's four lanes are all inside or all outside
  const int64_t first = (int64_t)blockIdx.x * (U * kThreads8) + threadIdx.x;
  Vec8<T> v[U];
  Item it[U];
  Walk<kWhole> walk;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    it[u] = walk.next(u, first + u * kThreads8, items, vp, v8, row);
    if (it[u].real) v[u].load(x, it[u].vec);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    // magnitudes compare as their bits do; infinities and NaN are above the rest
    uint32_t top = it[u].real ? v[u].top() : 0u;
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // e + 127: m / 2^e is in [64, 128) for e = ⌊log₂ m⌋ − 6, and one more is needed from 127.5 on,
    // which rint takes to 128
    int e = (int)(top >> 23) - 6;
    if (e >= 0 && __uint_as_float(top) * __uint_as_float((uint32_t)(254 - e) << 23) >= 127.5f) ++e;
    e = min(max(e, 0), kTopScale);
    const bool finite = top < kInfBits;
    const float inv = finite ? __uint_as_float((uint32_t)(254 - e) << 23) : 0.0f;
    if (first + u * kThreads8 < items && (threadIdx.x & 3) == 0) scales[it[u].group] = finite ? (uint8_t)e : (uint8_t)255;
    if (!it[u].real) continue;
    if (e == kTopScale) v[u].hold();  // (changes nothing below 127.5·2^121)
    float f[8];
    v[u].get(f);
    // x / 2^e plus 1.5·2^23 in one rounding is rint(x / 2^e) in the last bits of the sum
    uint32_t r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = __float_as_uint(fmaf(f[j], inv, 12582912.0f));
    const uint32_t lo = __byte_perm(__byte_perm(r[0], r[1], 0x0040), __byte_perm(r[2], r[3], 0x0040), 0x5410);
    const uint32_t hi = __byte_perm(__byte_perm(r[4], r[5], 0x0040), __byte_perm(r[6], r[7], 0x0040), 0x5410);
    codes[it[u].vec] = finite ? make_uint2(lo, hi) : make_uint2(0u, 0u);
  }
}

template <typename T, bool kWhole>
__global__ void __launch_bounds__(kThreads8)
    act8_unpack_kernel(const uint2* __restrict__ codes, const uint8_t* __restrict__ scales, void* __restrict__ x,
                       int64_t items, int vp, int v8, RowOf row, bool wide) {
  constexpr int U = kItems<T>;
  const int64_t first = (int64_t)blockIdx.x * (U * kThreads8) + threadIdx.x;
  Item it[U];
  uint2 w[U];
  uint32_t e[U];
  Walk<kWhole> walk;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    it[u] = walk.next(u, first + u * kThreads8, items, vp, v8, row);
    if (it[u].real) {
      w[u] = __ldcs(codes + it[u].vec);
      e[u] = scales[it[u].group];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!it[u].real) continue;
    // 2^(e − 127): e = 0 is subnormal
    const float step = e[u] == 255u ? __uint_as_float(0x7FC00000u)
                                    : __uint_as_float(e[u] > 0u ? e[u] << 23 : 1u << 22);
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = (float)(int8_t)((j < 4 ? w[u].x : w[u].y) >> (8 * (j % 4))) * step;
    Vec8<T>::store(x, it[u].vec, f, wide);
  }
}

}  // namespace

cudaError_t launch_act8_pack(const void* x, void* codes, void* scales, int64_t rows, int C, bool bf16,
                             cudaStream_t s) {
  const bool whole = C % kGroup == 0;
  const int v8 = C / 8, vp = (C + kGroup - 1) / kGroup * 4;
  const int64_t items = rows * vp;
  const int per_block = kThreads8 * (bf16 ? kItems<__nv_bfloat16> : kItems<float>);
  const int64_t blocks = (items + per_block - 1) / per_block;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  auto kern = bf16 ? (whole ? act8_pack_kernel<__nv_bfloat16, true> : act8_pack_kernel<__nv_bfloat16, false>)
                   : (whole ? act8_pack_kernel<float, true> : act8_pack_kernel<float, false>);
  kern<<<(unsigned)blocks, kThreads8, 0, s>>>(x, static_cast<uint2*>(codes), static_cast<uint8_t*>(scales), items, vp,
                                              v8, row_of(vp / 4));
  return cudaGetLastError();
}

cudaError_t launch_act8_unpack(const void* codes, const void* scales, void* x, int64_t rows, int C, bool bf16,
                               cudaStream_t s) {
  const bool whole = C % kGroup == 0;
  const int v8 = C / 8, vp = (C + kGroup - 1) / kGroup * 4;
  const int64_t items = rows * vp;
  const int per_block = kThreads8 * (bf16 ? kItems<__nv_bfloat16> : kItems<float>);
  const int64_t blocks = (items + per_block - 1) / per_block;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  auto kern = bf16 ? (whole ? act8_unpack_kernel<__nv_bfloat16, true> : act8_unpack_kernel<__nv_bfloat16, false>)
                   : (whole ? act8_unpack_kernel<float, true> : act8_unpack_kernel<float, false>);
  kern<<<(unsigned)blocks, kThreads8, 0, s>>>(static_cast<const uint2*>(codes), static_cast<const uint8_t*>(scales),
                                              x, items, vp, v8, row_of(vp / 4), (reinterpret_cast<uintptr_t>(x) & 31u) == 0);
  return cudaGetLastError();
}

}  // namespace rglru
