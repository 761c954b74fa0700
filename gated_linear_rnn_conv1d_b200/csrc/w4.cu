// Linears with 4-bit weights for a few tokens, for serving: y = x Ŵᵀ and the gated pair
// h = act(x Ŵ_gᵀ) ⊙ (x Ŵ_uᵀ), x [M][K] bf16 with M ≤ 64,
//     Ŵ[n][k] = s[n][k / G] · (q[n][k] − 8),   q in 4 bits (even k in the low half of a byte), s bf16.
// HBM's floor is half a byte a weight and 2 / G of scale. The kernel is few_tokens.cuh's. Up to eight tokens latency
// bounds it: 52 MB take 15.3 µs (3.4 TB/s; alone and cold 20.4, HBM at a third of its rate and the issue slots at 40 %:
// 22 instructions a warp for 256 weights, eleven the unpacking and two the products, are 7.6 µs of them), and warps wait
// for loads as much as for anything else; a ring of two steps has one in flight. More tokens than 16 cost more than
// their bytes (16, 32 and 64 tokens 19, 36 and 67 µs; the bf16 block, with four times the bytes, 37, 44 and 52).
#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>

#include "few_tokens.cuh"
#include "kernels.cuh"

namespace rglru {
namespace {

template <int GROUP, bool GLU, int ACT> cudaError_t launch_group(const FewArgs& a, cudaStream_t s) {
  using F = FewW4<GROUP>;
  // A chunk takes all of a block's granules where it can: x and its order are then formed once, and a ring step of
  // up to three granules has its bookkeeping once. K = 4096, G = 128, eight tokens, chunks of 1, 2, 3
  // and 6 granules: one granule a block (4096 rows) 3.9, 4.3, 4.5 and 4.9 µs; two (8192) 6.6, 5.6, 5.7 and 6.2;
  // three (12288) 9.6, 8.8, 6.9 and 7.5; five (20480) 15.0, 13.1, 11.4 and 9.8; sixteen tokens alike.
  const int granules = (a.rows + (GLU ? 7 : 15)) / (GLU ? 8 : 16);
  auto per = [&](int blocks) { return (granules + blocks - 1) / blocks; };
  if (a.M <= 16) {
    const int n = per(2 * num_sms());
    if (a.M <= 8)
      return n == 1   ? launch_few<F, GLU, ACT, 1, 1, 64, 1, 4>(a, s)
             : n == 2 ? launch_few<F, GLU, ACT, 1, 2, 64, 2, 2>(a, s)
             : n == 3 ? launch_few<F, GLU, ACT, 1, 3, 64, 3, 2>(a, s)
                      : launch_few<F, GLU, ACT, 1, 6, 64, 3, 2>(a, s);
    return n == 1   ? launch_few<F, GLU, ACT, 2, 1, 64, 1, 4>(a, s)
           : n == 2 ? launch_few<F, GLU, ACT, 2, 2, 64, 2, 2>(a, s)
           : n == 3 ? launch_few<F, GLU, ACT, 2, 3, 64, 3, 2>(a, s)
                    : launch_few<F, GLU, ACT, 2, 6, 64, 3, 2>(a, s);
  }
  // Up to 32 tokens one block an SM (4096 rows 7.1 and 8.4 µs for chunks of 2 and 6, 8192 rows 13.4 and 11.3); more
  // tokens are two halves, each of half the blocks (12288 gated channels, 64 tokens: 68 µs, and 133 with
  // all their sums in one block's registers).
  return per(num_sms()) <= 2 ? launch_few<F, GLU, ACT, 4, 2, 64, 2, 4>(a, s)
                             : launch_few<F, GLU, ACT, 4, 6, 64, 3, 3>(a, s);
}

template <bool GLU, int ACT> cudaError_t launch_any(const FewArgs& a, int group, cudaStream_t s) {
  switch (group) {
    case 32: return launch_group<32, GLU, ACT>(a, s);
    case 64: return launch_group<64, GLU, ACT>(a, s);
    case 128: return launch_group<128, GLU, ACT>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

FewArgs few_args(const W4Matrix& w0, const W4Matrix& w1, const void* x, void* out, int M, int rows, int K,
                 int group) {
  FewArgs a{};
  a.row_groups = K / group;
  a.out_ld = rows;
  a.w0 = static_cast<const uint8_t*>(w0.codes);
  a.w1 = static_cast<const uint8_t*>(w1.codes);
  a.scales0 = static_cast<const __nv_bfloat16*>(w0.scales);
  a.scales1 = static_cast<const __nv_bfloat16*>(w1.scales);
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.row_bytes = K / 2;
  a.M = M;
  a.rows = rows;
  a.K = K;
  return a;
}

// Quantisation, once for a matrix: a thread forms one group of one row (12288 × 4096: 76 µs in groups of 128, 47 in groups
// of 32, of 19 that HBM's rate asks for: neighbouring threads read a group's width apart). s = bf16(max |w| / 7), q = rint(w / s) + 8, the
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
  return launch_any<false, kActGelu>(few_args(w, w, x, y, M, rows, K, group), group, s);
}

cudaError_t launch_w4_glu(const W4Matrix& gate, const W4Matrix& up, const void* x, void* h, int M, int rows, int K,
                          int group, int act, cudaStream_t s) {
  const FewArgs a = few_args(gate, up, x, h, M, rows, K, group);
  return act == kActGelu ? launch_any<true, kActGelu>(a, group, s) : launch_any<true, kActSilu>(a, group, s);
}

}  // namespace rglru
