// Attention of the 8-bit path: device helpers and host-side launchers (gfx950 / CDNA4, wave64).
#pragma once

#include "kq_fp8.hpp"

namespace kq {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// 32 x 32 x 16 and 16 x 16 x 32 products of 16-bit fragments (eight values a lane), float32 sums.
template <bool BF16>
__device__ __forceinline__ v16f mfma32(const v4u& a, const v4u& b, const v16f& c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

template <bool BF16>
__device__ __forceinline__ v4f mfma16(const v4u& a, const v4u& b, const v4f& c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// Four rows of sixteen 16-bit values, transposed within each 16 lanes: lane i gives the address of values
// 4 (i % 4) .. + 3 of row (i % 16) / 4 and gets value i % 16 of the four rows.
__device__ __forceinline__ v2u lds_tr16(const void* p) {
  typedef __attribute__((address_space(3))) v4s lds_v4s;
  return __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)p));
}

// Eight rows of sixteen bytes, likewise: lane i gives the address of bytes 8 (i % 2) .. + 7 of row
// (i % 16) / 2 and gets byte i % 16 of the eight rows.
__device__ __forceinline__ v2u lds_tr8(const void* p) {
  typedef int v2i __attribute__((ext_vector_type(2)));
  typedef __attribute__((address_space(3))) v2i lds_v2i;
  return __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i*)p));
}

// The other half of the wavefront's value, joined.
__device__ __forceinline__ float half_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Narrows [lo, lo + len) to at most 64 candidates for the last i with before(i), which holds up to some i and for none
// behind it: 64 samples at a time.  (Whatever `before` says, the candidates stay within the given range.)
template <class F>
__device__ __forceinline__ void narrow(int& lo, int& len, F before) {
  const int lane = threadIdx.x & 63;
  while (len > 64) {
    const int step = (len + 63) / 64;
    const int c = __popcll(__ballot(lane * step < len && before(lo + lane * step)));
    const int skip = c > 1 ? (c - 1) * step : 0;
    lo += skip;
    len = min(step, len - skip);
  }
}

// The last i of [0, n) with before(i) (0 where it holds for none), the same in every lane.
template <class F>
__device__ __forceinline__ int last_before(int n, F before) {
  int lo = 0, len = n;
  narrow(lo, len, before);
  const int lane = threadIdx.x & 63, c = __popcll(__ballot(lane < len && before(lo + min(lane, len - 1))));
  return __builtin_amdgcn_readfirstlane(lo + (c > 0 ? c - 1 : 0));
}

// Rows of heads: element (token, head, d) at p[token * ts + head * hs + d].
struct AttnRows {
  const uint8_t* p;
  int64_t ts, hs;                      // in bytes
};

struct AttnArgs {
  AttnRows q, k, v;
  const int32_t *cu_q, *cu_k;          // null: one sequence
  int64_t T, Tk;
  int32_t B, Hq, Hkv, D, causal;
  float c;                             // scale log2 e
  void* out;                           // [T][Hq][D], or codes [T][Hq * 128]
  uint8_t* scales;                     // with codes
  float* part;                         // workspace
  int32_t parts;                       // set by the launch
};
// 0: none needed
size_t attention_workspace_bytes(int64_t B, int64_t T, int64_t Tk, bool packed, int Hq, int Hkv, int D);
// precise: weights as sums of 16-bit numbers, with float32's precision
hipError_t launch_attention(bool bf16, bool precise, const AttnArgs& a, hipStream_t s);

// Pages of keys and values: head h's row r of a page at ((page * Hkv + h) * page_rows + r) * row bytes;
// scales (8-bit rows only) one byte a row, in the same order.
struct Pages {
  uint8_t *k, *v, *ks, *vs;
  const int32_t *table, *lengths;      // [B][width], [B]
  int64_t pages;
  int32_t B, width, page, Hkv, D;
};

struct PagedArgs {
  Pages c;
  const uint8_t* q;                    // element (b, head, d) at q + b * qs + head * qh, in bytes
  int64_t qs, qh;
  int32_t Hq;
  float scale;                         // scale log2 e
  void* out;                           // [B][Hq][D], or codes [B][Hq * 128]
  uint8_t* scales;                     // with codes
  float* part;                         // workspace
};
size_t paged_workspace_bytes(int64_t B, int Hq, int Hkv, int D, int64_t longest);
// wide: 16-bit rows of the queries' type; else E4M3
hipError_t launch_paged_attention(bool bf16, bool wide, const PagedArgs& a, hipStream_t s);

struct AppendArgs {
  Pages c;
  AttnRows k, v;
  const int32_t* cu;                   // null: one token a sequence
  int64_t T;
};
hipError_t launch_cache_append(bool bf16, bool wide, const AppendArgs& a, hipStream_t s);

}  // namespace kq
