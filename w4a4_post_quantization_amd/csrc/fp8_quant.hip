// 8-bit activations: E4M3 codes with one E8M0 scale for every 128 consecutive values.
//   quantize:  y = x
//   norm:      h = x + residual, y = h / sqrt(mean_k h^2 + eps) * gamma_k
// then per group of 128: e the smallest exponent with max|y| <= 448 2^e, code = E4M3(y 2^-e).
// Both read each input once and write each output once, so HBM bounds them; a wavefront takes
// 512 columns at a time (16-byte loads, one dword of scale bytes), and the norm's row stays in
// registers between its sum and its output.
#include "kq_fp8.hpp"
#include "kq_launch.hpp"

namespace kq {

// KIND: 0 fp16, 1 bf16, 2 float32.  Units of 512 columns, numbered along the rows, U
// consecutive ones per wavefront and step.
template <int KIND, int U>
__global__ __launch_bounds__(256) void f8_quantize_kernel(const uint8_t* __restrict__ X, int64_t M, int K,
                                                          uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int lane = threadIdx.x & 63;
  const int segs = (K + 511) / 512;
  const int64_t total = M * segs;
  const int64_t nw = (int64_t)gridDim.x * 4;
  for (int64_t u = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * U; u < total; u += nw * U) {
    int64_t row[U];
    int col[U];
    v4u raw[U][KIND == 2 ? 2 : 1];
    row[0] = total <= 0x7FFFFFFF ? (int64_t)((uint32_t)u / (uint32_t)segs) : u / segs;
    int seg = (int)(u - row[0] * segs);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (i > 0) {
        row[i] = row[i - 1];
        if (++seg == segs) seg = 0, ++row[i];
      }
      col[i] = u + i < total ? 512 * seg + 8 * lane : K;       // K: nothing to load or store
#pragma unroll
      for (int p = 0; p < (KIND == 2 ? 2 : 1); ++p) {
        raw[i][p] = v4u{0, 0, 0, 0};
        if (col[i] < K)
          raw[i][p] = *reinterpret_cast<const v4u*>(X + (row[i] * K + col[i]) * (KIND == 2 ? 4 : 2) + 16 * p);
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float y[8];
      if (KIND == 2) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t w = raw[i][j / 4][j % 4];
          y[j] = __uint_as_float(w);
        }
      } else {
        unpack8_16<KIND == 1>(raw[i][0], y);
      }
      f8_store_512(y, row[i], col[i], K, lane, codes, scales);
    }
  }
}

template <int KIND, int U>
static hipError_t quantize_go(const void* X, int64_t M, int64_t K, uint8_t* codes, uint8_t* scales, hipStream_t s) {
  int64_t grid = (M * ((K + 511) / 512) + 4 * U - 1) / (4 * U);
  if (grid > (1 << 20)) grid = 1 << 20;
  hipLaunchKernelGGL((f8_quantize_kernel<KIND, U>), dim3((unsigned)grid), dim3(256), 0, s,
                     static_cast<const uint8_t*>(X), M, (int)K, codes, scales);
  return hipGetLastError();
}

// Four units a wavefront for their loads in flight, one where a few workgroups would be left: 385 units
// 2.1 us with one and 3.0 with four, 4096 2.9 and 3.2, 8192 3.75 and 3.73, 32768 9.45 and 8.82.
template <int KIND>
static hipError_t quantize_launch(const void* X, int64_t M, int64_t K, uint8_t* codes, uint8_t* scales, hipStream_t s) {
  return M * ((K + 511) / 512) <= 4096 ? quantize_go<KIND, 1>(X, M, K, codes, scales, s)
                                       : quantize_go<KIND, 4>(X, M, K, codes, scales, s);
}

hipError_t launch_f8_quantize(bool bf16, const void* X, int64_t M, int64_t K, uint8_t* codes, uint8_t* scales,
                              hipStream_t s) {
  return bf16 ? quantize_launch<1>(X, M, K, codes, scales, s) : quantize_launch<0>(X, M, K, codes, scales, s);
}

hipError_t launch_f8_quantize_f32(const float* X, int64_t M, int64_t K, uint8_t* codes, uint8_t* scales,
                                  hipStream_t s) {
  return quantize_launch<2>(X, M, K, codes, scales, s);
}

// 1 / sqrt(x) from the hardware's estimate (good to a step) by one Newton step in float64: with the
// sum joined in float64 too, the factor of a whole row is off by its own rounding alone.
__device__ __forceinline__ float f8_rsqrt(double x) {
  const double r = (double)__builtin_amdgcn_rsqf((float)x);
  return (float)fma(0.5 * r, fma(-x * r, r, 1.0), r);
}

// The sum over a workgroup's threads, the same bits in each.
template <int NT>
__device__ __forceinline__ double f8_block_sum(double sum, double* part, int t) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
  if ((t & 63) == 0) part[t >> 6] = sum;
  __syncthreads();
  sum = part[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) sum += part[w];
  return sum;
}

// One row per NT threads at a time; thread t holds columns 8 (v NT + t) .. + 7 for v < VPT in
// float32.  h is normalized as summed in float32; only the stored residual is rounded to 16 bits.
// A lane's squares are a float32 chain, the lanes' sums are joined in float64.  Rows whose squares may
// have left float32's range (bf16 reaches 3e38) take them again in float64, and their factor, which
// may itself be out of float32's range, in two parts.
template <bool BF16, bool RES, int NT, int VPT>
__global__ __launch_bounds__(NT) void f8_rmsnorm_kernel(const uint8_t* __restrict__ X,
                                                        const uint8_t* residual,
                                                        const uint8_t* __restrict__ gamma, float eps, int64_t M, int K,
                                                        uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                        uint8_t* residual_out) {
  const int t = threadIdx.x, lane = t & 63;
  __shared__ double part[NT / 64];
  for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
    float h[VPT][8];
    float sq = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int col = 8 * (v * NT + t);
      v4u a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
      if (col < K) {
        a = *reinterpret_cast<const v4u*>(X + (row * K + col) * 2);
        if (RES) b = *reinterpret_cast<const v4u*>(residual + (row * K + col) * 2);
      }
      unpack8_16<BF16>(a, h[v]);
      if (RES) {
        float r[8];
        unpack8_16<BF16>(b, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[v][i] += r[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sq = fmaf(h[v][i], h[v][i], sq);
    }
    double mean = f8_block_sum<NT>((double)sq, part, t) / (double)K + (double)eps;
    float rinv;
    int ex = 0;                                                // h 2^ex rinv is the normalized row
    // squares below 2^-126 count for nothing beside 2^-100; NaN comes here too
    if (__builtin_expect(mean >= 0x1p-100 && mean <= 0x1p100, 1)) {
      rinv = f8_rsqrt(mean);
    } else {
      double sq64 = 0.0;
#pragma unroll
      for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) sq64 = fma((double)h[v][i], (double)h[v][i], sq64);
      __syncthreads();                                         // part has been read
      mean = f8_block_sum<NT>(sq64, part, t) / (double)K + (double)eps;
      const double r = 1.0 / sqrt(mean);
      rinv = (float)r;
      if (r > 0.0 && r < INFINITY) rinv = (float)frexp(r, &ex);
    }
    ex = __builtin_amdgcn_readfirstlane(ex);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int col = 8 * (v * NT + t);
      if (512 * ((v * NT + t) >> 6) >= K) break;               // the whole wavefront is past the row
      v4u gw = {0, 0, 0, 0};
      if (col < K) {
        gw = *reinterpret_cast<const v4u*>(gamma + col * 2);
        if (RES) {
          const v4u o = {pack2_16<BF16>(h[v][0], h[v][1]), pack2_16<BF16>(h[v][2], h[v][3]),
                         pack2_16<BF16>(h[v][4], h[v][5]), pack2_16<BF16>(h[v][6], h[v][7])};
          *reinterpret_cast<v4u*>(residual_out + (row * K + col) * 2) = o;
        }
      }
      float g[8], y[8];
      unpack8_16<BF16>(gw, g);
      // lanes past K: 0 times a possibly infinite rinv is not to reach the group's maximum
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = h[v][i];
      if (__builtin_expect(ex != 0, 0)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = ldexpf(y[i], ex);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = col < K ? y[i] * rinv * g[i] : 0.0f;
      f8_store_512(y, row, col, K, lane, codes, scales);
    }
    __syncthreads();                                           // part is read before the next row's
  }
}

template <bool BF16, bool RES>
static void rmsnorm_launch(const uint8_t* X, const uint8_t* residual, const uint8_t* gamma, float eps, int64_t M, int K,
                           uint8_t* codes, uint8_t* scales, uint8_t* out, hipStream_t s) {
  const dim3 g((unsigned)(M < (1 << 22) ? M : 1 << 22));       // a launch is at most 2^32 threads
#define KQ_NORM(NT, VPT)                                                                                             \
  hipLaunchKernelGGL((f8_rmsnorm_kernel<BF16, RES, NT, VPT>), g, dim3(NT), 0, s, X, residual, gamma, eps, M, K, codes, \
                     scales, out)
  if (K <= 2048) KQ_NORM(256, 1);
  else if (K <= 4096) KQ_NORM(256, 2);
  else if (K <= 8192) KQ_NORM(256, 4);
  else KQ_NORM(256, 8);
#undef KQ_NORM
}

hipError_t launch_f8_rmsnorm(bool bf16, const void* X, const void* residual, const void* gamma, float eps, int64_t M,
                             int64_t K, uint8_t* codes, uint8_t* scales, void* residual_out, hipStream_t s) {
  const uint8_t* x = static_cast<const uint8_t*>(X);
  const uint8_t* r = static_cast<const uint8_t*>(residual);
  const uint8_t* g = static_cast<const uint8_t*>(gamma);
  uint8_t* o = static_cast<uint8_t*>(residual_out);
  if (bf16 && r) rmsnorm_launch<true, true>(x, r, g, eps, M, (int)K, codes, scales, o, s);
  else if (bf16) rmsnorm_launch<true, false>(x, r, g, eps, M, (int)K, codes, scales, o, s);
  else if (r) rmsnorm_launch<false, true>(x, r, g, eps, M, (int)K, codes, scales, o, s);
  else rmsnorm_launch<false, false>(x, r, g, eps, M, (int)K, codes, scales, o, s);
  return hipGetLastError();
}

}  // namespace kq
