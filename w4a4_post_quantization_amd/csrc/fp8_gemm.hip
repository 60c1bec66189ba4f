// The 8-bit linear: Y = Xq Wq^T (+ bias), and the gated pair H = act(Xq Wg^T) * (Xq Wu^T).
// Both operands are E4M3 with one E8M0 scale per row and 128 consecutive k:
//   y[m][n] = sum_g 2^(ex[m][g] + ew[n][g]) sum_{k in g} qx[m][k] qw[n][k],
// which is what the scaled matrix instruction v_mfma_scale_f32_32x32x64_f8f6f4 computes when
// each lane is given its row's scale byte.  The order of k inside a group is free as long as
// both operands use the same one, so a lane takes 32 consecutive bytes of its row.
#include "kq_fp8.hpp"
#include "kq_launch.hpp"

namespace kq {

// act: 0 SiLU, 1 GELU, 2 GELU's tanh form, which is g / (1 + exp -2z) without tanh's cancellation.
// GELU's g Phi(g) goes through erfc for the same reason.
__device__ __forceinline__ float f8_act(int act, float g) {
  if (act == 1) return 0.5f * g * erfcf(-0.70710678118654752f * g);
  const float x = act == 0 ? g : 1.5957691216057308f * fmaf(0.044715f * g * g, g, g);
  return g / (1.0f + expf(-x));
}

// 64 x 64 output tile, 2 x 2 wavefronts of 32 x 32, operands straight from global memory.
template <bool GATED, bool BF16>
__global__ __launch_bounds__(256) void f8_simple_kernel(const uint8_t* __restrict__ wcodes,
                                                        const uint8_t* __restrict__ wscales,
                                                        const uint8_t* __restrict__ xcodes,
                                                        const uint8_t* __restrict__ xscales, int64_t M, int N, int K,
                                                        const uint16_t* __restrict__ bias, void* __restrict__ out,
                                                        int act) {
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int l32 = lane & 31, h = lane >> 5;
  const int SC = (int)f8_scale_cols(K);
  const int n0 = blockIdx.x * 64 + (wid & 1) * 32;
  const int64_t m0 = (int64_t)blockIdx.y * 64 + (wid >> 1) * 32;
  const int n = n0 + l32;
  const int64_t m = m0 + l32;
  v16f acc[GATED ? 2 : 1];
#pragma unroll
  for (int t = 0; t < (GATED ? 2 : 1); ++t)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[t][e] = 0.0f;
  auto load = [&](const uint8_t* row, bool live, int k) {
    v4i lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
    if (live && k < K) lo = *reinterpret_cast<const v4i*>(row + k);
    if (live && k + 16 < K) hi = *reinterpret_cast<const v4i*>(row + k + 16);
    return v8i{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  };
  for (int k0 = 0; k0 < K; k0 += 64) {
    const int k = k0 + 32 * h, g = k0 >> 7;
    const v8i b = load(xcodes + m * K, m < M, k);
    const int sb = m < M ? xscales[m * SC + g] : 0;
#pragma unroll
    for (int t = 0; t < (GATED ? 2 : 1); ++t) {
      const int64_t r = n + (int64_t)t * N;
      const v8i a = load(wcodes + r * K, n < N, k);
      const int sa = n < N ? wscales[r * SC + g] : 0;
      acc[t] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc[t], 0, 0, 0, sa, 0, sb);
    }
  }
  if (m >= M) return;
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const int col = n0 + 8 * (q >> 2) + 4 * h + (q & 3);
    if (col >= N) continue;
    float v = acc[0][q];
    if (GATED) {
      static_cast<float*>(out)[m * N + col] = f8_act(act, v) * acc[GATED ? 1 : 0][q];
    } else {
      if (bias) v += unpack1_16<BF16>(bias[col]);
      static_cast<uint16_t*>(out)[m * N + col] = (uint16_t)pack2_16<BF16>(v, 0.0f);
    }
  }
}

static dim3 simple_grid(int64_t M, int64_t N) { return dim3((unsigned)((N + 63) / 64), (unsigned)((M + 63) / 64)); }

size_t f8_linear_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_f8_linear(bool bf16, const uint8_t* xcodes, const uint8_t* xscales, int64_t M, int64_t K,
                            const uint8_t* wcodes, const uint8_t* wscales, int64_t N, const void* bias, void* Y,
                            void* workspace, hipStream_t s) {
  const uint16_t* b = static_cast<const uint16_t*>(bias);
  if (bf16)
    hipLaunchKernelGGL((f8_simple_kernel<false, true>), simple_grid(M, N), dim3(256), 0, s, wcodes, wscales, xcodes,
                       xscales, M, (int)N, (int)K, b, Y, 0);
  else
    hipLaunchKernelGGL((f8_simple_kernel<false, false>), simple_grid(M, N), dim3(256), 0, s, wcodes, wscales, xcodes,
                       xscales, M, (int)N, (int)K, b, Y, 0);
  return hipGetLastError();
}

size_t f8_gated_workspace_bytes(int64_t M, int64_t F, int64_t) { return (size_t)M * F * 4; }

hipError_t launch_f8_gated(int act, const uint8_t* xcodes, const uint8_t* xscales, int64_t M, int64_t K,
                           const uint8_t* wcodes, const uint8_t* wscales, int64_t F, uint8_t* codes, uint8_t* scales,
                           void* workspace, hipStream_t s) {
  hipLaunchKernelGGL((f8_simple_kernel<true, false>), simple_grid(M, F), dim3(256), 0, s, wcodes, wscales, xcodes,
                     xscales, M, (int)F, (int)K, nullptr, workspace, act);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_f8_quantize_f32(static_cast<const float*>(workspace), M, F, codes, scales, s);
}

}  // namespace kq
