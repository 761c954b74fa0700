// The gated feed-forward block for a few tokens, its forward (serving) and dg, du and h of its backward: h = act(x W_gᵀ) ⊙ (x W_uᵀ) with
// x [N][D], N ≤ 32, bf16 weights streamed once by few_tokens.cuh's kernel.
#include <cstdint>
#include <cuda_bf16.h>

#include "few_tokens.cuh"
#include "kernels.cuh"

namespace rglru {
namespace {
// The copies are two to four granules ahead. 201 MB of weights, eight tokens: chunks of 1, 2, 3 and 6 granules 34.2,
// 32.4, 32.0 and 33.0 µs (a chunk shares the loads of x, which are read through what shared memory leaves of
// the L1); sixteen: 33.3 and 33.8 for 2 and 3; 24: 38.2 and 37.9; 32, in steps of two granules and of one: 38.0 and
// 43.5 (three granules a block, 6144 channels of 2048, in one chunk: 11.7 and 13.4). The tiles of 256 rows (glu.cu) take
// 42 µs for 17 tokens to 64; of 34 MB, D 4096, H 2048, they take 16 and this 9 for 24 tokens and 10 for 32.
template <int ACT, bool GRAD> cudaError_t launch_act(const FewArgs& a, cudaStream_t s) {
  const int n = (a.rows / 8 + 2 * num_sms() - 1) / (2 * num_sms());  // granules of a block
  return a.M <= 8    ? launch_few<FewBf16, true, ACT, 1, 3, 128, 1, 5, GRAD>(a, s)
         : a.M <= 16 ? launch_few<FewBf16, true, ACT, 2, 2, 128, 1, 4, GRAD>(a, s)
         : a.M <= 24 ? launch_few<FewBf16, true, ACT, 3, 3, 128, 1, 3, GRAD>(a, s)
         : n == 3    ? launch_few<FewBf16, true, ACT, 4, 3, 128, 1, 3, GRAD>(a, s)
                     : launch_few<FewBf16, true, ACT, 4, 2, 128, 2, 2, GRAD>(a, s);
}
FewArgs few_args(const void* W_gate, const void* W_up, const void* x, void* out, int64_t N, int D, int H) {
  FewArgs a{};
  a.w0 = static_cast<const uint8_t*>(W_gate);
  a.w1 = static_cast<const uint8_t*>(W_up);
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.row_bytes = (int64_t)D * 2;
  a.M = (int)N;
  a.rows = a.out_ld = H;
  a.K = D;
  return a;
}
}  // namespace

cudaError_t launch_glu_few(const void* W_gate, const void* W_up, const void* x, void* h, int N, int D, int H, int act,
                           cudaStream_t s) {
  const FewArgs a = few_args(W_gate, W_up, x, h, N, D, H);
  return act == kActGelu ? launch_act<kActGelu, false>(a, s) : launch_act<kActSilu, false>(a, s);
}

cudaError_t launch_glu_few_grad(const GluBwdArgs& b, cudaStream_t s) {
  FewArgs a = few_args(b.W_gate, b.W_up, b.x, b.dg, b.N, b.D, b.H);
  a.out_ld = glu_scratch_pitch(b.H);
  a.dh = static_cast<const __nv_bfloat16*>(b.dh);
  a.du = static_cast<__nv_bfloat16*>(b.du);
  a.h = static_cast<__nv_bfloat16*>(b.h);
  return b.act == kActGelu ? launch_act<kActGelu, true>(a, s) : launch_act<kActSilu, true>(a, s);
}

}  // namespace rglru
