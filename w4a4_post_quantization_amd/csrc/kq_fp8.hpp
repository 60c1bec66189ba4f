// E4M3 values with one E8M0 scale for every 128 consecutive values: device helpers and
// host-side launchers of the 8-bit path (gfx950 / CDNA4, wave64).
#pragma once

#include "kq_device.hpp"

namespace kq {

constexpr int F8_GROUP = 128;

// Bytes of a row of scales: one per group, padded with zero bytes to whole dwords.
__host__ __device__ constexpr int64_t f8_scale_cols(int64_t K) { return (K + 511) / 512 * 4; }

// E8M0 byte of a group from the bits of its largest magnitude: the smallest power of two 2^e
// with a <= 448 2^e (448 = 1.75 2^8 is E4M3's largest value), so no value saturates.  A
// power of two costs an element nothing: E4M3's precision is relative.  Zero and magnitudes
// below 448 2^-127 take byte 0; an infinity or NaN takes 255, the format's NaN.
__device__ __forceinline__ uint32_t f8_scale_byte(uint32_t abits) {
  const uint32_t ef = abits >> 23;
  if (ef == 255u) return 255u;
  const uint32_t e = ef + ((abits & 0x7FFFFFu) > 0x600000u ? 1u : 0u);
  return e > 8u ? e - 8u : 0u;
}

// 2^-e for a scale byte below 255 (exponents 6 .. 254: always a normal float).
__device__ __forceinline__ float f8_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Four float32 values times inv -> four E4M3 codes (round to nearest even).  |v inv| <= 448.
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d, float inv) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}

// Largest magnitude, as float bits (which order like the magnitudes, NaN above infinity).
__device__ __forceinline__ uint32_t umax32(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Max over the 16 lanes of a DPP row (every lane of the row gets the result).
__device__ __forceinline__ uint32_t row16_umax(uint32_t v) {
  v = umax32(v, dpp_u<0x128>(v));                       // row_ror:8
  v = umax32(v, dpp_u<0x124>(v));                       // row_ror:4
  v = umax32(v, dpp_u<quad_perm(2, 3, 0, 1)>(v));
  return umax32(v, dpp_u<quad_perm(1, 0, 3, 2)>(v));
}

// Eight 16-bit values (fp16 or bf16) -> float32, and back with rounding to nearest even.
template <bool BF16>
__device__ __forceinline__ void unpack8_16(const v4u& raw, float* x) {
  if (BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = raw[i];
      x[2 * i] = __uint_as_float(w << 16);
      x[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
    }
  } else {
    unpack8_f16(raw, x);
  }
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2_16(float a, float b) {
  if (BF16) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    const b2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
  }
  return __builtin_bit_cast(uint32_t, __floats2half2_rn(a, b));
}

template <bool BF16>
__device__ __forceinline__ float unpack1_16(uint16_t w) {
  return BF16 ? __uint_as_float((uint32_t)w << 16) : __half2float(__ushort_as_half(w));
}

// A wavefront's 512 consecutive columns (lane l holds columns 8 l .. 8 l + 7, so each DPP row
// of 16 lanes is one group): codes and the dword with the four scale bytes.  `col` is the
// lane's first column; lanes past K hold zeros and store nothing.
__device__ __forceinline__ void f8_store_512(const float* y, int64_t row, int col, int K, int lane,
                                             uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = umax32(a, abs_bits(y[i]));
  const uint32_t byte = f8_scale_byte(row16_umax(a));
  const bool bad = byte == 255u;
  const float inv = bad ? 1.0f : f8_inv_scale(byte);
  uint2 q;
  q.x = bad ? 0x7F7F7F7Fu : f8_pack4(y[0], y[1], y[2], y[3], inv);
  q.y = bad ? 0x7F7F7F7Fu : f8_pack4(y[4], y[5], y[6], y[7], inv);
  if (col < K) *reinterpret_cast<uint2*>(codes + row * K + col) = q;
  const uint32_t b0 = __builtin_amdgcn_readlane(byte, 0), b1 = __builtin_amdgcn_readlane(byte, 16);
  const uint32_t b2 = __builtin_amdgcn_readlane(byte, 32), b3 = __builtin_amdgcn_readlane(byte, 48);
  if (lane == 0 && col < K)
    *reinterpret_cast<uint32_t*>(scales + row * f8_scale_cols(K) + (col >> 7)) = b0 | (b1 << 8) | (b2 << 16) | (b3 << 24);
}

// X [M][K] fp16 (bf16: bf16) -> codes [M][K], scales [M][f8_scale_cols(K)].
hipError_t launch_f8_quantize(bool bf16, const void* X, int64_t M, int64_t K, uint8_t* codes, uint8_t* scales,
                              hipStream_t s);
// The same from float32 rows (the gated product's intermediate).
hipError_t launch_f8_quantize_f32(const float* X, int64_t M, int64_t K, uint8_t* codes, uint8_t* scales,
                                  hipStream_t s);
// h = X + residual (residual may be null), residual_out = round(h), codes/scales of
// h / sqrt(mean h^2 + eps) * gamma.
hipError_t launch_f8_rmsnorm(bool bf16, const void* X, const void* residual, const void* gamma, float eps, int64_t M,
                             int64_t K, uint8_t* codes, uint8_t* scales, void* residual_out, hipStream_t s);

// precise: products of the exact codes summed in float32 whatever the number of tokens
hipError_t launch_f8_linear(bool bf16, bool precise, const uint8_t* xcodes, const uint8_t* xscales, int64_t M, int64_t K,
                            const uint8_t* wcodes, const uint8_t* wscales, int64_t N, const void* bias, void* Y,
                            hipStream_t s);
size_t f8_gated_workspace_bytes(int64_t M, int64_t F, int64_t K);
// act: 0 SiLU, 1 GELU (erf), 2 GELU (tanh)
hipError_t launch_f8_gated(int act, bool precise, const uint8_t* xcodes, const uint8_t* xscales, int64_t M, int64_t K,
                           const uint8_t* wcodes, const uint8_t* wscales, int64_t F, uint8_t* codes, uint8_t* scales,
                           void* workspace, hipStream_t s);

}  // namespace kq
