// The 8-bit linear: Y = Xq Wq^T (+ bias), and the gated pair H = act(Xq Wg^T) * (Xq Wu^T).
// Both operands are E4M3 with one E8M0 scale per row and 128 consecutive k:
//   y[m][n] = sum_g 2^(ex[m][g] + ew[n][g]) sum_{k in g} qx[m][k] qw[n][k],
// which is what the scaled matrix instruction v_mfma_scale_f32_32x32x64_f8f6f4 computes when
// each lane is given its row's scale byte.  The order of k inside a group is free as long as
// both operands use the same one, so a lane takes 32 consecutive bytes of its row.
#include "kq_fp8.hpp"
#include "kq_launch.hpp"

#include <algorithm>

namespace kq {

// act: 0 SiLU, 1 GELU, 2 GELU's tanh form, which is g / (1 + exp -2z) without tanh's cancellation.
// GELU's g Phi(g) goes through erfc for the same reason.  Beside 8-bit products (not WIDE) the
// exponential is the hardware's exp2, whose rounded argument moves the result by up to |x| 2^-24, and
// the quotient its reciprocal: the library's forms cost five times as many instructions, and the
// products before them are good to 1e-5 and the result is rounded to four bits next.
template <int ACT, bool WIDE>
__device__ __forceinline__ float f8_act(float g) {
  if (WIDE && ACT == 0) return g / (1.0f + expf(-g));
  if (WIDE && ACT == 2) return g / (1.0f + expf(-1.5957691216057308f * fmaf(0.044715f * g * g, g, g)));
  if (ACT == 1) return 0.5f * g * erfcf(-0.70710678118654752f * g);
  constexpr float L = 1.4426950408889634f;              // log2 e
  const float x = ACT == 0 ? -L * g : -1.5957691216057308f * L * fmaf(0.044715f * g * g, g, g);
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x));
}

// ---------------------------------------------------------------------------------
// Few tokens (up to 16 MT): the weights' bytes bound it.  A workgroup takes 16 RT weight rows
// (gated: 16 gate rows and the 16 up rows of the same columns) and all tokens; its NW
// wavefronts take the 128-wide groups of k in turn and their sums are added through LDS in
// wavefront order.  Each wavefront streams its groups through a ring of S slots of its own in
// LDS, so the loop has no barrier: 8 rows x 128 bytes a load, whole cache lines.  (Loading the
// fragments straight into registers puts a different row in every lane; the address unit then
// takes one lane a cycle, 64 cycles instead of 16 a load, which bound it: 4096 x 11008 by one
// token 10.3 us, 6144 x 4096 by 64 tokens 28.8 us.)  A row's eight 16-byte chunks are
// XOR-swizzled by the row; lane l holds row l % 16 and chunks l / 16 and 4 + l / 16 of it, the
// same k for both operands.  Scale bytes of 128 groups (16384 k) at a time are staged for all.
// WIDE: the codes are widened to bf16 with their scale applied (exact: four significant bits)
// and multiplied by the bf16 matrix instruction, which sums in float32.  The 8-bit instruction
// cuts each of eight consecutive products off, towards zero, at 2^(E - 13), E the largest of their sums of
// two exponents (norm of the errors over norm of the sums 1.0e-5 to 1.6e-5 on Gaussian values, to 7e-5 with
// outlier channels; WIDE 1e-8 to 2e-7).  For up to 16 tokens there is time under the loads to do without
// that; above, the caller chooses.  Measured (us) 8-bit and WIDE: linear 6144 x 4096, 17 tokens 7.7 and 7.7,
// 37 8.2 and 8.5, 64 9.6 and 10.1; gated 11008 x 4096, 32 tokens 20.3 and 20.9; in tiles, 4096 tokens: linear 4096 x
// 11008 144 and 308, gated 11008 x 4096 309 and 645 (bf16 instructions at half the rate, and no 256 x 256 tiles:
// the widened fragments beside 256 accumulators exceed the registers).
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));

// Eight of the sixteen codes in a piece (P = 0, 1), widened and scaled.
template <int P>
__device__ __forceinline__ v8b f8_widen8(const v4i& w, float scale) {
  const uint32_t lo = (uint32_t)w[2 * P], hi = (uint32_t)w[2 * P + 1];
  const v2b a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const v2b b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const v2b c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const v2b d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return v8b{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// acc + one 32 x 32 block's products of 64 k, 32 codes a lane; the order of k is the lanes' own.
template <bool WIDE>
__device__ __forceinline__ v16f f8_product(const v8i& a, const v8i& b, const v16f& acc, int sa, int sb) {
  if constexpr (!WIDE) return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc, 0, 0, 0, sa, 0, sb);
  const v4i a0 = {a[0], a[1], a[2], a[3]}, a1 = {a[4], a[5], a[6], a[7]};
  const v4i b0 = {b[0], b[1], b[2], b[3]}, b1 = {b[4], b[5], b[6], b[7]};
  const float fa = __uint_as_float((uint32_t)sa << 23), fb = __uint_as_float((uint32_t)sb << 23);
  v16f c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f8_widen8<0>(a0, fa), f8_widen8<0>(b0, fb), acc, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f8_widen8<1>(a0, fa), f8_widen8<1>(b0, fb), c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f8_widen8<0>(a1, fa), f8_widen8<0>(b1, fb), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(f8_widen8<1>(a1, fa), f8_widen8<1>(b1, fb), c, 0, 0, 0);
}

template <int ACT, bool BF16, bool WIDE, int RT, int MT, int NW, int S>   // ACT -1: the linear
__global__ __launch_bounds__(64 * NW) void f8_rows_kernel(const uint8_t* __restrict__ wcodes,
                                                          const uint8_t* __restrict__ wscales,
                                                          const uint8_t* __restrict__ xcodes,
                                                          const uint8_t* __restrict__ xscales, int M, int N, int K,
                                                          const uint16_t* __restrict__ bias, void* __restrict__ out) {
  constexpr bool GATED = ACT >= 0;
  constexpr int NF = RT + MT;                                  // 16-row fragments of a group: RT weight, MT token
  constexpr int SLOT = 2048 * NF, RING = NW * S * SLOT, SCALES = 2048 * NF, PART = NW * RT * MT * 1024;
  static_assert(!GATED || RT == 2, "gate and up");
  __shared__ __align__(16) uint8_t lds[(RING > PART ? RING : PART) + SCALES];
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int SC = (int)f8_scale_cols(K), T = (K + 127) / 128;
  const int n0 = 16 * (GATED ? 1 : RT) * blockIdx.x;
  v4i rc[NF], rs[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int64_t row = f < RT ? n0 + (int64_t)f * (GATED ? N : 16) : 16 * (f - RT);
    const int64_t rows = f < RT ? (GATED ? 16 : min(16, N - n0 - 16 * f)) : min(16, M - 16 * (f - RT));
    rc[f] = rsrc_words((f < RT ? wcodes : xcodes) + row * K, rows * K);
    rs[f] = rsrc_words((f < RT ? wscales : xscales) + row * SC, rows * SC);
  }
  const uint32_t lds0 = lds_addr(lds), ring0 = lds0 + wid * S * SLOT;
  const int lr = lane >> 3, lc = 16 * ((lane & 7) ^ lr);       // a load's row (+ 8) and chunk of this lane
  auto load = [&](int slot, int t) {                           // group t (past the last: zeros)
    const int k = 128 * t + lc;
    const uint32_t off = t < T && k < K ? lr * K + k : KQ_OOB;
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int p = 0; p < 2; ++p) lds_load16(rc[f], ring0 + slot * SLOT + 2048 * f + 1024 * p, (int)(off + 8 * p * K));
  };
  const int sw = r & 7, c0 = 128 * r + 16 * (q ^ sw), c1 = 128 * r + 16 * ((4 + q) ^ sw);
  v4f acc[RT][MT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  constexpr int SC_OFF = RING > PART ? RING : PART;
  int slot = 0, t = wid;
  for (int t1 = 0; t1 < T; t1 += 128) {                        // 16384 k: one round for all but the longest
    __syncthreads();
    for (int f = wid; f < 2 * NF; f += NW) {                   // 8 rows of scale bytes a load
      const uint32_t at = lr * SC + t1 + lc;
      v4i src = rs[0];
#pragma unroll
      for (int e = 1; e < NF; ++e) src = f / 2 == e ? rs[e] : src;
      lds_load16(src, lds0 + SC_OFF + 1024 * f, (int)(at + 8 * (f & 1) * SC));
    }
    if (t1 == 0) {
#pragma unroll
      for (int u = 0; u < S; ++u) load(u, t + u * NW);
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(S * 2 * NF));      // the scales
    } else {
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    }
    lds_barrier();
    const int t2 = min(T, t1 + 128);
    for (; t < t2; t += NW) {
      __builtin_amdgcn_s_waitcnt(waitcnt_vm((S - 1) * 2 * NF));
      asm volatile("" ::: "memory");
      const uint8_t* const st = lds + wid * S * SLOT + slot * SLOT;
      const int ts = t - t1;
      const uint8_t* const sc = lds + SC_OFF + 128 * r + 16 * ((ts >> 4) ^ sw) + (ts & 15);
      v4i lo[NF], hi[NF];
      int s[NF];
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        lo[f] = *reinterpret_cast<const v4i*>(st + 2048 * f + c0);
        hi[f] = *reinterpret_cast<const v4i*>(st + 2048 * f + c1);
        s[f] = sc[2048 * f];
      }
      // the slot is free once its fragments are in registers
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      load(slot, t + S * NW);
      __builtin_amdgcn_sched_barrier(0);
      slot = slot + 1 == S ? 0 : slot + 1;
      if constexpr (WIDE) {
        v8b xb[MT][4];
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          const float sx = __uint_as_float((uint32_t)s[RT + j] << 23);
          xb[j][0] = f8_widen8<0>(lo[RT + j], sx);
          xb[j][1] = f8_widen8<1>(lo[RT + j], sx);
          xb[j][2] = f8_widen8<0>(hi[RT + j], sx);
          xb[j][3] = f8_widen8<1>(hi[RT + j], sx);
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const float sw = __uint_as_float((uint32_t)s[i] << 23);
          const v8b w[4] = {f8_widen8<0>(lo[i], sw), f8_widen8<1>(lo[i], sw), f8_widen8<0>(hi[i], sw), f8_widen8<1>(hi[i], sw)};
#pragma unroll
          for (int p = 0; p < 4; ++p)
#pragma unroll
            for (int j = 0; j < MT; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[p], xb[j][p], acc[i][j], 0, 0, 0);
        }
      } else {
        auto join = [&](int f) { return v8i{lo[f].x, lo[f].y, lo[f].z, lo[f].w, hi[f].x, hi[f].y, hi[f].z, hi[f].w}; };
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int i = 0; i < RT; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(i), join(RT + j), acc[i][j], 0, 0, 0, s[i], 0, s[RT + j]);
      }
    }
  }
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));                   // the last refills, before the ring is reused
  __syncthreads();
  v4f* const part = reinterpret_cast<v4f*>(lds);               // [NW][RT MT][64]
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) part[(wid * RT * MT + i * MT + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  // 16 tokens (gated) or 16 x 16 outputs a wavefront at a time: lane l holds columns
  // 4 (l / 16) .. + 3 of token l % 16
  for (int f = wid; f < (GATED ? MT : RT * MT); f += NW) {
    v4f s[2];
#pragma unroll
    for (int i = 0; i < (GATED ? 2 : 1); ++i) {
      s[i] = part[(i * MT + f) * 64 + lane];
#pragma unroll
      for (int v = 1; v < NW; ++v) s[i] += part[(v * RT * MT + i * MT + f) * 64 + lane];
    }
    const int m = 16 * (f % MT) + r, col = n0 + 16 * (GATED ? 0 : f / MT) + 4 * q;
    if (m >= M || col >= N) continue;
    if constexpr (GATED) {
      v4f y;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = f8_act<ACT, WIDE>(s[0][e]) * s[1][e];
      *reinterpret_cast<v4f*>(static_cast<float*>(out) + (int64_t)m * N + col) = y;
    } else {
      if (bias) {
        const uint2 b = *reinterpret_cast<const uint2*>(bias + col);
        s[0][0] += unpack1_16<BF16>((uint16_t)(b.x & 0xFFFFu));
        s[0][1] += unpack1_16<BF16>((uint16_t)(b.x >> 16));
        s[0][2] += unpack1_16<BF16>((uint16_t)(b.y & 0xFFFFu));
        s[0][3] += unpack1_16<BF16>((uint16_t)(b.y >> 16));
      }
      uint2 o;
      o.x = pack2_16<BF16>(s[0][0], s[0][1]);
      o.y = pack2_16<BF16>(s[0][2], s[0][3]);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + (int64_t)m * N + col) = o;
    }
  }
}

template <int ACT, bool BF16, bool WIDE, int RT, int MT, int NW, int S>
static hipError_t rows_go(const uint8_t* xcodes, const uint8_t* xscales, int64_t M, int64_t K, const uint8_t* wcodes,
                          const uint8_t* wscales, int64_t N, const uint16_t* bias, void* out, hipStream_t s) {
  const int64_t per = ACT >= 0 ? 16 : 16 * RT;
  hipLaunchKernelGGL((f8_rows_kernel<ACT, BF16, WIDE, RT, MT, NW, S>), dim3((unsigned)((N + per - 1) / per)), dim3(64 * NW), 0,
                     s, wcodes, wscales, xcodes, xscales, (int)M, (int)N, (int)K, bias, out);
  return hipGetLastError();
}

// Tokens the rows kernel takes with this many workgroups of 32 weight rows: to 32, and to 48 and 64 while the
// workgroups all run at once, three and two on a compute unit; else, and above, tiles.  The linear, measured (us)
// in rows and in tiles on 256 compute units: 4096 k, 64 tokens, 6144 rows 9.0 and 11.1, 16384 14.7 and 14.0, 18432 23.8
// and 17.3, 28672 37.0 and 34.2; 40 tokens, 16384 14.4 and 13.5, 22016 21.3 and 23.7, 24576 26.9 and 30.6, 28672 35.1
// and 33.4; 32 tokens, 22016 22.7 and 24.3, 57344 52.5 and 58.1; 8192 k, 64 tokens, 18432 59.7 and 52.7, 40 tokens, 24576
// 47.4 and 56.1, 28672 60.7 and 56.0; 128 tokens of 6144 rows, 4096 k, 13.1 and 12.3.
static bool rows_fit(int64_t M, int64_t wgs) {
  const int64_t cus = device_cu_count();
  return M <= 32 || (M <= 48 && wgs <= 3 * cus) || (M <= 64 && wgs <= 2 * cus);
}

// The gated pair, whose second launch and float32 outputs between them count too.  Measured (us) in rows and in
// tiles, 256 compute units, K = 4096: 40 tokens, F = 2816 12.7 and 18.6, 11008 23.3 and 25.9, 14336 36.7 and 33.0; 64
// tokens, 2816 13.4 and 19.0, 8192 17.2 and 19.3, 11008 32.2 and 26.5; 32 tokens, 14336 33.2 and 33.0.
static bool gated_rows(int64_t M, int64_t F) { return rows_fit(M, F / 16); }

template <int ACT, bool BF16>
static hipError_t rows_launch(bool precise, const uint8_t* xcodes, const uint8_t* xscales, int64_t M, int64_t K,
                              const uint8_t* wcodes, const uint8_t* wscales, int64_t N, const uint16_t* bias,
                              void* out, hipStream_t s) {
#define KQ_ROWS(RT, MT, NW, S) \
  (precise || MT == 1 ? rows_go<ACT, BF16, true, RT, MT, NW, S> : rows_go<ACT, BF16, (MT == 1), RT, MT, NW, S>)(xcodes, xscales, M, K, wcodes, wscales, N, bias, out, s)
  if constexpr (ACT >= 0) {
    // two workgroups on a compute unit; one of twice the LDS took 20.7 against 17.7 us (one token, 11008 x
    // 4096) and 22.6 against 19.0 (32 tokens)
    if (M <= 32) return M <= 16 ? KQ_ROWS(2, 1, 4, 3) : KQ_ROWS(2, 2, 4, 2);
    return M <= 48 ? KQ_ROWS(2, 3, 2, 2) : KQ_ROWS(2, 4, 2, 2);
  } else {
    // 16 weight rows a workgroup while that is at most one workgroup per compute unit, with twice the
    // wavefronts if one token leaves some idle (2048 x 11008: 6.5 against 7.3 us); else 32, which halves
    // what the tokens' codes cost, in workgroups small enough for two or three on a unit.  Measured (us)
    // with 16 and 32 rows, weights from HBM: one token, 11008 x 4096 13.8 and 12.3, 5120 x 6144 9.6 and
    // 8.1, but 8192 x 8192 14.6 and 18.8; 24 tokens, 11008 x 4096 16.0 and 13.9, 4096 x 4096 7.1 and 7.8.
    // Two wavefronts instead of four once 32 rows a workgroup are more than one per unit: 37
    // tokens, 16384 x 4096 17.3 against 20.3, 6144 x 4096 10.3 against 9.4.
    const int64_t wgs = (N + 15) / 16, cus = device_cu_count();
    if (M <= 16) {
      if (wgs < cus) return KQ_ROWS(1, 1, 8, 2);
      return wgs > cus && K <= 6144 ? KQ_ROWS(2, 1, 4, 3) : KQ_ROWS(1, 1, 4, 4);
    }
    if (M <= 32) return wgs <= cus ? KQ_ROWS(1, 2, 4, 2) : KQ_ROWS(2, 2, 4, 2);
    if (M <= 48) return wgs <= cus ? KQ_ROWS(1, 3, 4, 2) : wgs <= 2 * cus ? KQ_ROWS(2, 3, 4, 2) : KQ_ROWS(2, 3, 2, 2);
    return wgs <= cus ? KQ_ROWS(1, 4, 4, 2) : wgs <= 2 * cus ? KQ_ROWS(2, 4, 4, 2) : KQ_ROWS(2, 4, 2, 2);
  }
#undef KQ_ROWS
}

// ---------------------------------------------------------------------------------
// Middling token counts, linear: tiles of 64 TN weight rows by 64 TM token rows on four wavefronts
// (2 x 2), each TN x TM blocks of 32 x 32.  The operands go from
// global memory straight into LDS, 64 k (one matrix instruction) a stage, NS stages deep; a
// stage's row is four 16-byte chunks, XOR-swizzled so that the fragment reads (16 rows x one
// chunk) and the staging writes hit distinct banks.  Lane l of half h = l / 32 takes chunks h
// and 2 + h of its row as its 32 values of k.
// A step is G stages: wait for the next step's loads, one barrier, which makes them visible and
// frees this step's slots (its fragments are in registers), then this step's products, with the
// reads of the next step's fragments and the loads that refill the freed slots spread between
// them.  Large tiles have enough products in one stage; for small ones a step of one stage would
// be the latency of its fragment reads.
// Scale bytes come 16 at a time for each row (2048 k, so seldom) into a double-buffered area.
template <int TN_, int TM_, int NS_, int G_>
struct F8Small {
  static constexpr int TN = TN_, TM = TM_, NS = NS_, G = G_;
  static constexpr int BN = 64 * TN, BM = 64 * TM;
  static constexpr int A_BYTES = BN * 64, STAGE = A_BYTES + BM * 64;
  static constexpr int SC_OFF = NS * STAGE;                    // two sets of 16 groups' bytes, BN + BM rows
  static constexpr int SC_BYTES = (BN + BM) * 16;
  static constexpr int BIAS_OFF = SC_OFF + 2 * SC_BYTES;       // 64 lanes x 16 bytes (BN biases used)
  static constexpr int LDS = BIAS_OFF + 1024;
};

__device__ __forceinline__ int f8_swz(int row) { return ((row >> 1) ^ (row >> 2)) & 3; }

// Weight rows n0 .. n0 + BN - 1, token rows m0 .. m0 + BM - 1.
template <bool BF16, bool WIDE, class C>
__device__ __forceinline__ void f8_small_tile(uint8_t* __restrict__ lds, const uint8_t* __restrict__ wcodes,
                                              const uint8_t* __restrict__ wscales, const uint8_t* __restrict__ xcodes,
                                              const uint8_t* __restrict__ xscales, int64_t M, int N, int K,
                                              const uint16_t* __restrict__ bias, uint8_t* __restrict__ out, int64_t m0,
                                              int n0) {
  constexpr int NS = C::NS, TN = C::TN, TM = C::TM, G = C::G;
  constexpr int NA = TN, NB = TM, NL = NA + NB;                // loads (16 rows) of a wave and stage
  constexpr int NR = 2 * (TN + TM);                            // reads of 64 k
  const int tid = threadIdx.x;
  const int lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wid & 1, wm = wid >> 1;
  const int l32 = lane & 31, h = lane >> 5;
  const int SC = (int)f8_scale_cols(K);
  const int T = (K + 127) / 128;                               // groups (zeros past K)

  // wave w stages weight rows 16 NA w .. of the tile and token rows 16 NB w ..; the first waves also
  // the scales of 64 rows each
  const v4i rA = rsrc_words(wcodes + (int64_t)(n0 + 16 * NA * wid) * K, (int64_t)(N - n0 - 16 * NA * wid) * K);
  const v4i rAS = rsrc_words(wscales + (int64_t)(n0 + 64 * wid) * SC, (int64_t)(N - n0 - 64 * wid) * SC);
  const int64_t mleft = min(M - m0, (int64_t)C::BM);
  const v4i rB = rsrc_words(xcodes + m0 * K, mleft * K);
  const v4i rBS = rsrc_words(xscales + m0 * SC, mleft * SC);

  const uint32_t lds0 = lds_addr(lds);
  const int lrow = lane >> 2, lcol = 16 * ((lane & 3) ^ f8_swz(lrow));   // a load's row and first byte of this lane
  // unsigned: an offset past the end is KQ_OOB plus at most 2^28 and stays past every range
  const uint32_t ogA = lrow * K, ogB = (16 * NB * wid + lrow) * K;
  auto k_off = [&](int ks) -> uint32_t { return 64 * ks + lcol < K ? 64 * ks + lcol : KQ_OOB; };
  auto code_load = [&](int slot, uint32_t ko, int g) {         // load g (0 .. NL - 1) of a stage
    const uint32_t st = lds0 + (uint32_t)(slot * C::STAGE);
    if (g < NA) lds_load16(rA, st + (16 * NA * wid + 16 * g) * 64, (int)(ogA + 16 * g * K + ko));
    else lds_load16(rB, st + C::A_BYTES + (16 * NB * wid + 16 * (g - NA)) * 64, (int)(ogB + 16 * (g - NA) * K + ko));
  };
  // scale bytes of groups 16 grp .. 16 grp + 15, issued only when skip is zero, by the waves that
  // have rows: the branches are inside the assembly so that the loop body stays one block for
  // the scheduler.  A row's last piece may run into the next row; those bytes are never read.
  const uint32_t osc = lane * SC, oscb = (64 * wid + lane) * SC;
  auto scale_loads = [&](int grp, int skip) {
    const uint32_t sc = lds0 + (uint32_t)(C::SC_OFF + (grp & 1) * C::SC_BYTES + 16 * 64 * wid);
    const uint32_t ko = 16 * grp < T ? 16 * grp : KQ_OOB;
    asm volatile(
        "s_cmp_lg_u32 %0, 0\n\t"
        "s_cbranch_scc1 1f\n\t"
        "s_mov_b32 m0, %2\n\t"
        "buffer_load_dwordx4 %4, %6, 0 offen lds\n"
        "1:\n\t"
        "s_cmp_lg_u32 %1, 0\n\t"
        "s_cbranch_scc1 2f\n\t"
        "s_mov_b32 m0, %3\n\t"
        "buffer_load_dwordx4 %5, %7, 0 offen lds\n"
        "2:"
        :: "s"(__builtin_amdgcn_readfirstlane(wid < TN ? skip : 1)),
           "s"(__builtin_amdgcn_readfirstlane(wid < TM ? skip : 1)), "s"(__builtin_amdgcn_readfirstlane(sc)),
           "s"(__builtin_amdgcn_readfirstlane(sc + C::BN * 16)), "v"(osc + ko), "v"(oscb + ko), "s"(rAS), "s"(rBS)
        : "memory", "m0", "scc");
  };

  const int wrow_a = 32 * TN * wn, wrow_b = 32 * TM * wm;
  const int sw = f8_swz(l32);                                  // the same for every block of 32 rows
  const int fa = (wrow_a + l32) * 64, fb = C::A_BYTES + (wrow_b + l32) * 64;
  const int c0 = 16 * (h ^ sw), c1 = 16 * ((2 + h) ^ sw);
  auto read_half = [&](const uint8_t* st, int q, v8i* a, v8i* b) {   // half fragment q (0 .. NR - 1)
    const int f = q >> 1;
    const v4i v = *reinterpret_cast<const v4i*>(st + (f < TN ? fa + 2048 * f : fb + 2048 * (f - TN)) + ((q & 1) ? c1 : c0));
    v8i& d = f < TN ? a[f] : b[f - TN];
#pragma unroll
    for (int e = 0; e < 4; ++e) d[4 * (q & 1) + e] = v[e];
  };
  const int sa_at = 16 * (wrow_a + l32), sb_at = C::BN * 16 + 16 * (wrow_b + l32);
  auto read_scale = [&](int grp, int q) -> int {               // scale of fragment q for a group of k
    const uint8_t* sc = lds + C::SC_OFF + ((grp >> 4) & 1) * C::SC_BYTES + (grp & 15);
    return sc[q < TN ? sa_at + 512 * q : sb_at + 512 * (q - TN)];
  };

  v16f acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  if (wid == 0) {                                    // without a bias, or past N: zeros
    const v4i rW = rsrc_words(bias + n0, bias ? (int64_t)(N - n0) * 2 : 0);
    lds_load16(rW, lds0 + C::BIAS_OFF, lane < C::BN / 8 ? 16 * lane : KQ_OOB);
  }
  scale_loads(0, 0);
#pragma unroll
  for (int p = 0; p < NS; ++p)
#pragma unroll
    for (int g = 0; g < NL; ++g) code_load(p, k_off(p), g);
  static_assert(G == 1 || G == 2, "a loop body of two steps is whole groups");
  static_assert(NS % (2 * G) == 0, "the two steps of a loop body never wrap inside the ring");
  constexpr int NM = G * TN * TM;
  const int nk = 2 * T;                                      // stages
  __builtin_amdgcn_s_waitcnt(waitcnt_vm((NS - G) * NL));     // biases, scales and the first step's stages
  lds_barrier();
  v8i a[2][G][TN], b[2][G][TM];
  int s[2][TN + TM];                                         // G = 1: the first set for both steps
#pragma unroll
  for (int q = 0; q < TN + TM; ++q) s[0][q] = read_scale(0, q);
#pragma unroll
  for (int q = 0; q < G * NR; ++q) read_half(lds + q / NR * C::STAGE, q % NR, a[0][q / NR], b[0][q / NR]);

  int slot = 0, after = 2 * G % NS;                          // of stages ks and ks + 2 G
  for (int ks = 0; ks < nk; ks += 2 * G) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // the next step's stages have landed once at most those of the NS - 2 G behind them are
      // outstanding
      const int k0 = ks + u * G;
      __builtin_amdgcn_s_waitcnt(waitcnt_vm((NS - 2 * G) * NL));
      lds_barrier();
      __builtin_amdgcn_sched_barrier(0);
      // the next step's fragments, and its scales if it starts a group
      auto reads = [&](int q0, int q1) {
#pragma unroll
        for (int q = q0; q < q1; ++q)
          read_half(lds + ((u == 0 ? slot + G : after) + q / NR) * C::STAGE, q % NR, a[1 - u][q / NR], b[1 - u][q / NR]);
      };
      auto scales = [&](int q0, int q1) {
#pragma unroll
        for (int q = q0; q < q1; ++q) s[G == 1 ? 1 : 1 - u][q] = read_scale((k0 + G) / 2, q);
      };
      if (G > 1) {
        reads(0, G * NR);
        scales(0, TN + TM);
        __builtin_amdgcn_sched_barrier(0);
      }
      uint32_t ko[G];
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        const int c = m / (TN * TM), i = m / TM % TN, j = m % TM;
        const int* const sc = s[G == 1 ? 0 : u];
        // behind the last group the codes are zeros, and no scale byte found there may be NaN
        const int on = G == 1 || k0 + c < nk ? -1 : 0;
        acc[i][j] = f8_product<WIDE>(a[u][c][i], b[u][c][j], acc[i][j], sc[i] & on, sc[TN + j] & on);
        __builtin_amdgcn_sched_barrier(0);
        if (m == 0) {
          if (u == 0) scale_loads((ks >> 5) + 1, ks & 31);
#pragma unroll
          for (int d = 0; d < G; ++d) ko[d] = k_off(k0 + NS + d);
        }
        if (G == 1) {
          reads(NR * m / NM, NR * (m + 1) / NM);
          if (u == 1) scales((TN + TM) * m / NM, (TN + TM) * (m + 1) / NM);
        }
#pragma unroll
        for (int g = G * NL * m / NM; g < G * NL * (m + 1) / NM; ++g) code_load(slot + u * G + g / NL, ko[g / NL], g % NL);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (G == 1) {
#pragma unroll
      for (int q = 0; q < TN + TM; ++q) s[0][q] = s[1][q];
    }
    slot = after;
    after = after + 2 * G == NS ? 0 : after + 2 * G;
  }
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));                   // no load may land in LDS after this tile

  const __amdgpu_buffer_rsrc_t rY = make_rsrc(out + m0 * N * 2, mleft * N * 2);
  const uint32_t* const bias_t = reinterpret_cast<const uint32_t*>(lds + C::BIAS_OFF);
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int ml = wrow_b + 32 * j + l32;
#pragma unroll
    for (int i = 0; i < TN; ++i) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        uint32_t pk[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int g = 2 * p + u;
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * g + e];
          const uint32_t* const w = bias_t + (wrow_a + 32 * i + 8 * g + 4 * h) / 2;
          const uint32_t w01 = w[0], w23 = w[1];
          v[0] += unpack1_16<BF16>((uint16_t)(w01 & 0xFFFFu));
          v[1] += unpack1_16<BF16>((uint16_t)(w01 >> 16));
          v[2] += unpack1_16<BF16>((uint16_t)(w23 & 0xFFFFu));
          v[3] += unpack1_16<BF16>((uint16_t)(w23 >> 16));
          pk[u][0] = pack2_16<BF16>(v[0], v[1]);
          pk[u][1] = pack2_16<BF16>(v[2], v[3]);
        }
        // a lane holds columns 8 g + 4 h .. + 3: one lane-half swap per dword leaves lanes
        // 0 .. 31 with the eight columns of group 2 p and the others with those of 2 p + 1
        const auto s0 = __builtin_amdgcn_permlane32_swap(pk[0][0], pk[1][0], false, false);
        const auto s1 = __builtin_amdgcn_permlane32_swap(pk[0][1], pk[1][1], false, false);
        const v4i outv = {(int)s0[0], (int)s1[0], (int)s0[1], (int)s1[1]};
        const int col = n0 + wrow_a + 32 * i + 8 * (2 * p + h);
        __builtin_amdgcn_raw_buffer_store_b128(outv, rY, col < N ? (ml * N + col) * 2 : KQ_OOB, 0, 0);
      }
    }
  }
}

// Consecutive tile numbers, which the dispatcher deals out to the compute dies in turn, are
// remapped so that each die holds a contiguous run of tiles.
__device__ __forceinline__ int f8_remap(int pid, int n) {
  const int per = n / 8;
  return pid < 8 * per ? (pid % 8) * per + pid / 8 : pid;
}

// ---------------------------------------------------------------------------------
// Many tokens: tiles of 256 weight rows by 64 TM token rows on four wavefronts (2 x 2), each
// 128 x 32 TM as 4 x TM blocks of 32 x 32 (TM = 4: 256 float32 accumulators a lane).  A stage is
// 128 k, two matrix instructions deep, its rows eight 16-byte chunks, so that a load takes whole
// cache lines: 8 rows x 128 bytes.  With stages of 64 k each line is asked for twice, and with
// every compute unit at work the level-2 caches' request rate bound the loop (4096 x 4096 x 11008:
// 161 against 137 us).  Rows are XOR-swizzled so that the fragment reads hit distinct banks.
// A stage goes in two halves of 64 k, 4 TM products each.  First half: the second half's fragments
// are read under the first products; a barrier then frees the stage's slot, and half of the loads
// of the stage NS on go into it.  Second half: the other loads, and the next stage's first
// fragments, for which the wait and barrier between the halves made that stage visible.
// What bounds it: the chip's power.  In the loop the products take 2050 of 2300 (K = 4096) to
// 2550 (K = 11008) cycles of a whole tile's stage, at a clock of 1.67 to 1.78 GHz; alone on eight
// compute units the same loop runs at 2.4 GHz.
template <int TM_, int NS_>
struct F8Big {
  static constexpr int TM = TM_, BM = 64 * TM, NS = NS_;       // NS slots
  static constexpr int A_BYTES = 256 * 128, STAGE = A_BYTES + BM * 128;
  static constexpr int SC_OFF = NS * STAGE;                    // two sets of 16 groups' bytes, 256 + BM rows
  static constexpr int SC_BYTES = (256 + BM) * 16;
  static constexpr int BIAS_OFF = SC_OFF + 2 * SC_BYTES;       // 64 lanes x 16 bytes (256 biases used)
  static constexpr int TOP_OFF = BIAS_OFF + 1024;              // gated: 2 x BM maxima
  static constexpr int LDS = TOP_OFF + 2 * BM * 4;             // TM, NS = 4, 2: 150528 bytes; 2, 3: 161792
};

// The gated tiles' epilogue.  acc[0], acc[1] are gates, acc[2], acc[3] the up values of the
// same columns f0 + col0 + 32 i .., lane l's token of block j row0 + 32 j + l % 32.  Outputs in place
// of the gates, the maximum of each token's columns in this wave to LDS, and after the barrier the
// scale of all 128 (columns past F are zeros on both sides and stay zeros).
template <int ACT, bool WIDE, int TM>
__device__ __forceinline__ void f8_gated_store(v16f (&acc)[4][TM], uint8_t* __restrict__ lds_tops, int wn, int col0,
                                               int row0, int l32, int h, int64_t m0, int64_t mleft, int f0, int F,
                                               uint8_t* __restrict__ out, uint8_t* __restrict__ oscales) {
  uint32_t* const tops = reinterpret_cast<uint32_t*>(lds_tops);
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float v = f8_act<ACT, WIDE>(acc[i][j][e]) * acc[i + 2][j][e];
        acc[i][j][e] = v;
        top = umax32(top, abs_bits(v));
      }
    top = umax32(top, (uint32_t)__shfl_xor((int)top, 32, 64));
    if (h == 0) tops[64 * TM * wn + row0 + 32 * j + l32] = top;
  }
  lds_barrier();
  const int OS = (int)f8_scale_cols(F), grp = f0 >> 7;
  const __amdgpu_buffer_rsrc_t rQ = make_rsrc(out + m0 * F, mleft * F);
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int ml = row0 + 32 * j + l32;
    const uint32_t byte = f8_scale_byte(umax32(tops[ml], tops[64 * TM + ml]));
    const bool bad = byte == 255u;
    const float inv = bad ? 1.0f : f8_inv_scale(byte);
    if (wn == 0 && h == 0 && ml < mleft) {
      uint8_t* const row = oscales + (m0 + ml) * OS;
      row[grp] = (uint8_t)byte;
      if (f0 + 128 >= F)
        for (int q = grp + 1; q < OS; ++q) row[q] = 0;         // padding
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint32_t c = f8_pack4(acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3], inv);
        w[g] = bad ? 0x7F7F7F7Fu : c;
      }
      // dword g of half h is columns 8 g + 4 h .. + 3: swaps leave half h with 16 h .. + 15
      const auto s0 = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
      const auto s1 = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
      const v4i outv = {(int)s0[0], (int)s0[1], (int)s1[0], (int)s1[1]};
      const int col = f0 + col0 + 32 * i + 16 * h;
      __builtin_amdgcn_raw_buffer_store_b128(outv, rQ, col < F ? ml * F + col : KQ_OOB, 0, 0);
    }
  }
}

// ACT -1: the linear, weight rows n0 .. n0 + 255.  Gated: rows f0 .. f0 + 127 of both halves, f0 =
// n0 / 2, staged gate rows first; wavefront column wn takes gate and up of the same 64 columns, so
// that a lane has both factors of an output, and the tile's 128 columns are one scale group.
// at(t, m0, n0) gives tile t's place.  SEQ: the workgroup takes tiles t0, t0 + step, .. below end, and
// the loads past one tile's last stage are the next one's first: both slots of a gated tile, one of the
// linear's, whose outputs go through the other.  So only the first tile waits for memory.  T >= NS.
template <int ACT, bool BF16, bool WIDE, class C, bool SEQ, class At>
__device__ __forceinline__ void f8_big_tiles(uint8_t* __restrict__ lds, const uint8_t* __restrict__ wcodes,
                                            const uint8_t* __restrict__ wscales, const uint8_t* __restrict__ xcodes,
                                            const uint8_t* __restrict__ xscales, int64_t M, int N, int K,
                                            const uint16_t* __restrict__ bias, uint8_t* __restrict__ out,
                                            uint8_t* __restrict__ oscales, At at, int t0, int end, int step) {
  constexpr bool GATED = ACT >= 0;
  constexpr int NS = C::NS, TM = C::TM, NB = 2 * TM, NL = 8 + NB;   // NL loads (8 rows) of a wave and stage
  constexpr int NM = 4 * TM, NR = 2 * (4 + TM);                // products and reads of a half
  const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wid & 1, wm = wid >> 1;
  const int l32 = lane & 31, h = lane >> 5;
  const int SC = (int)f8_scale_cols(K), T = (K + 127) / 128;

  // wave w stages weight rows 64 w .. of the tile (gated: waves 0, 1 gate, 2, 3 up) and token rows
  // 8 NB w ..; the first waves also the scales of 64 token rows each
  auto rows_at = [&](int t, const uint8_t* w, const uint8_t* x, int stride, v4i& rw, v4i& rx) {
    int64_t m0;
    int n0;
    at(t < end ? t : t0, m0, n0);
    const int64_t row = GATED ? (int64_t)(wid >> 1) * N + (n0 >> 1) + 64 * (wid & 1) : (int64_t)n0 + 64 * wid;
    const int64_t left = GATED ? N - (n0 >> 1) - 64 * (wid & 1) : N - n0 - 64 * wid;
    rw = rsrc_words(w + row * stride, t < end ? left * stride : 0);   // no tile: nothing to load
    rx = rsrc_words(x + m0 * stride, t < end ? min(M - m0, (int64_t)C::BM) * stride : 0);
  };
  v4i rA, rB, rAS, rBS;
  auto codes_at = [&](int t) { rows_at(t, wcodes, xcodes, K, rA, rB); };
  auto scales_at = [&](int t) { rows_at(t, wscales, xscales, SC, rAS, rBS); };
  codes_at(t0);
  scales_at(t0);

  const uint32_t lds0 = lds_addr(lds);
  // a load's row and first byte of this lane; rows 8 .. 15 of each 16 have another swizzle
  const int lrow = lane >> 3, lcol = 16 * ((lane ^ lrow) & 7);
  // unsigned: an offset past the end is KQ_OOB plus at most 2^28 and stays past every range
  const uint32_t ogA = lrow * K, ogB = (8 * NB * wid + lrow) * K;
  auto k_off = [&](int k0, int odd) -> uint32_t {
    const int k = k0 + (lcol ^ (16 * odd));
    return k < K ? k : KQ_OOB;
  };
  auto code_load = [&](int slot, uint32_t ko, int g) {         // load g (0 .. NL - 1) of a stage
    const uint32_t st = lds0 + (uint32_t)(slot * C::STAGE);
    if (g < 8) lds_load16(rA, st + (64 * wid + 8 * g) * 128, (int)(ogA + 8 * g * K + ko));
    else lds_load16(rB, st + C::A_BYTES + (8 * NB * wid + 8 * (g - 8)) * 128, (int)(ogB + 8 * (g - 8) * K + ko));
  };
  // scale bytes of stages 16 grp .. 16 grp + 15, issued only when skip is zero, by the waves that
  // have rows: the branches are inside the assembly so that the loop body stays one block for
  // the scheduler.  A row's last piece may run into the next row; those bytes are never used.
  const uint32_t osc = lane * SC, oscb = (64 * wid + lane) * SC;
  int sbuf = 0;                                                // buffer of group 0 of this tile
  auto scale_loads = [&](int grp, int skip) {
    const uint32_t sc = lds0 + (uint32_t)(C::SC_OFF + ((sbuf + grp) & 1) * C::SC_BYTES + 16 * 64 * wid);
    const uint32_t ko = 16 * grp < T ? 16 * grp : SEQ ? 0 : KQ_OOB;
    asm volatile(
        "s_cmp_lg_u32 %0, 0\n\t"
        "s_cbranch_scc1 1f\n\t"
        "s_mov_b32 m0, %2\n\t"
        "buffer_load_dwordx4 %4, %6, 0 offen lds\n"
        "1:\n\t"
        "s_cmp_lg_u32 %1, 0\n\t"
        "s_cbranch_scc1 2f\n\t"
        "s_mov_b32 m0, %3\n\t"
        "buffer_load_dwordx4 %5, %7, 0 offen lds\n"
        "2:"
        :: "s"(__builtin_amdgcn_readfirstlane(skip)), "s"(__builtin_amdgcn_readfirstlane(wid < C::BM / 64 ? skip : 1)),
           "s"(__builtin_amdgcn_readfirstlane(sc)), "s"(__builtin_amdgcn_readfirstlane(sc + 256 * 16)), "v"(osc + ko),
           "v"(oscb + ko), "s"(rAS), "s"(rBS)
        : "memory", "m0", "scc");
  };

  // weight block i of a wavefront is staged row wrow_a + 32 blk(i) ..: gated blocks 0, 1 are its
  // gate rows, 2, 3 the up rows of the same columns, 128 rows on
  auto blk = [](int i) { return GATED ? 4 * (i >> 1) + (i & 1) : i; };
  const int wrow_a = (GATED ? 64 : 128) * wn, wrow_b = 32 * TM * wm;
  const int sw = (l32 ^ (l32 >> 3 & 1)) & 7;                   // the same for every block of 32 rows
  const int fa = (wrow_a + l32) * 128, fb = C::A_BYTES + (wrow_b + l32) * 128;
  // half fragment q (0 .. NR - 1) of half c of a stage: a lane's 32 values of the half's 64 k are
  // chunks h and 2 + h of its four
  auto read_half = [&](const uint8_t* st, int c, int q, v8i* a, v8i* b) {
    const int f = q >> 1, chunk = 16 * ((4 * c + 2 * (q & 1) + h) ^ sw);
    const v4i v = *reinterpret_cast<const v4i*>(st + (f < 4 ? fa + 4096 * blk(f) : fb + 4096 * (f - 4)) + chunk);
    v8i& d = f < 4 ? a[f] : b[f - 4];
#pragma unroll
    for (int e = 0; e < 4; ++e) d[4 * (q & 1) + e] = v[e];
  };
  const int sa_at = 16 * (wrow_a + l32), sb_at = 256 * 16 + 16 * (wrow_b + l32);
  auto read_scale = [&](int p, int q) -> int {                 // scale of fragment q for a stage
    const uint8_t* sc = lds + C::SC_OFF + ((sbuf + (p >> 4)) & 1) * C::SC_BYTES + (p & 15);
    return sc[q < 4 ? sa_at + 512 * blk(q) : sb_at + 512 * (q - 4)];
  };

  auto bias_load = [&](int n0) {
    if (!GATED && wid == 0) {                                  // without a bias, or past N: zeros
      const v4i rW = rsrc_words(bias + n0, bias ? (int64_t)(N - n0) * 2 : 0);
      lds_load16(rW, lds0 + C::BIAS_OFF, lane < 32 ? 16 * lane : KQ_OOB);
    }
  };
  {
    int64_t m0;
    int n0;
    at(t0, m0, n0);
    bias_load(n0);
  }
  scale_loads(0, 0);
#pragma unroll
  for (int p = 0; p < NS; ++p)
#pragma unroll
    for (int g = 0; g < NL; ++g) code_load(p, k_off(128 * p, g & 1), g);
  __builtin_amdgcn_s_waitcnt(waitcnt_vm((NS - 1) * NL));       // biases, scales and stage 0
  lds_barrier();
  int slot = 0, after = 1;                                     // of stages p and p + 1
  for (int t = t0;;) {
    v16f acc[4][TM];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    constexpr int ND = NM * 3 / 8, NE = NM * 3 / 4;            // products that the reads are spread under
    v8i a[2][4], b[2][TM];
    int s[4 + TM], ns[4 + TM];
#pragma unroll
    for (int q = 0; q < 4 + TM; ++q) s[q] = read_scale(0, q);
#pragma unroll
    for (int q = 0; q < NR; ++q) read_half(lds + slot * C::STAGE, 0, q, a[0], b[0]);
    int kb = 128 * NS;                                         // of the stage that is loaded
    const int e1 = (T - 1) & ~15, e2 = T - NS, ev = min(e1, e2);
    for (int p = 0; p < T; ++p, kb += 128) {
      if (SEQ && __builtin_expect(p >= ev, 0)) {               // from here on loads of the next tile
        if (p == e1) scales_at(t + step);
        if (p == e2) codes_at(t + step), kb = 0;
        if (!GATED && p > e2) kb = 1 << 20;                    // the outputs' slot
      }
      const uint8_t* const cur = lds + slot * C::STAGE;
      const uint8_t* const nxt = lds + after * C::STAGE;
      uint32_t ko[2];
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        const int i = m / TM, j = m % TM;
        acc[i][j] = f8_product<WIDE>(a[0][i], b[0][j], acc[i][j], s[i], s[4 + j]);
        __builtin_amdgcn_sched_barrier(0);
        if (m < ND) {
#pragma unroll
          for (int q = NR * m / ND; q < NR * (m + 1) / ND; ++q) read_half(cur, 1, q, a[1], b[1]);
        }
        if (m == NM / 2 - 1) {
          lds_barrier();
          scale_loads((p >> 4) + 1, p & 15);
          ko[0] = k_off(kb, 0);
          ko[1] = k_off(kb, 1);
        }
        if (m >= NM / 2) {
#pragma unroll
          for (int g = NL * (m - NM / 2) / NM; g < NL * (m + 1 - NM / 2) / NM; ++g) code_load(slot, ko[g & 1], g);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_waitcnt(waitcnt_vm((NS - 2) * NL + NL / 2));
      lds_barrier();
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        const int i = m / TM, j = m % TM;
        acc[i][j] = f8_product<WIDE>(a[1][i], b[1][j], acc[i][j], s[i], s[4 + j]);
        __builtin_amdgcn_sched_barrier(0);
        if (m < NE) {
#pragma unroll
          for (int q = NR * m / NE; q < NR * (m + 1) / NE; ++q) read_half(nxt, 0, q, a[0], b[0]);
#pragma unroll
          for (int q = (4 + TM) * m / NE; q < (4 + TM) * (m + 1) / NE; ++q) ns[q] = read_scale(p + 1, q);
        }
        if (m < NM / 2) {
#pragma unroll
          for (int g = NL / 2 + NL * m / NM; g < NL / 2 + NL * (m + 1) / NM; ++g) code_load(slot, ko[g & 1], g);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int q = 0; q < 4 + TM; ++q) s[q] = ns[q];
      slot = after;
      after = after + 1 == NS ? 0 : after + 1;
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));                 // no load may land in LDS after this tile
    int64_t m0;
    int n0;
    at(t, m0, n0);
    const int64_t mleft = min(M - m0, (int64_t)C::BM);
    // the lane, hidden from the compiler, which would keep the epilogue's addresses live in the loop
    int el = lane;
    asm volatile("" : "+v"(el));
    const int l32 = el & 31, h = el >> 5;

    if constexpr (!GATED) {
      // Outputs go through the slots, which a token's columns leave in whole cache lines: a lane
      // holds four columns of one token, and stored as they are the 64 lanes of a store touch 32
      // rows.  A wave's 32 TM tokens x 128 columns, rows of 16 chunks swizzled by the row, the halves
      // of a chunk swapped in rows 16 .. 31 of each 32 (a write's 32 lanes hit every bank).  (4096 x
      // 4096 x 1024: 23.4 against 29.4 us.)
      lds_barrier();                                           // every wave's loads have landed
      // SEQ: two of a wave's blocks of tokens at a time, in the slot that holds nothing
      constexpr int PJ = 2;
      uint8_t* const own = lds + (SEQ ? after * C::STAGE : 0) + wid * (32 * PJ * 256);
      const uint2* const bias_t = reinterpret_cast<const uint2*>(lds + C::BIAS_OFF);
      uint2 bw[4][4];                                          // all biases before the first use
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) bw[i][g] = bias_t[(wrow_a + 32 * i + 8 * g + 4 * h) / 4];
      const __amdgpu_buffer_rsrc_t rY = make_rsrc(out + m0 * N * 2, mleft * N * 2);
      const int c = el & 15, r4 = el >> 4, col = n0 + wrow_a + 8 * c;
      const uint32_t to = col < N ? ((uint32_t)(wrow_b + r4) * N + col) * 2 : KQ_OOB;
      const uint8_t* from[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) from[y] = own + (4 * y + r4) * 256 + 16 * (c ^ (4 * y + r4));
#pragma unroll
      for (int j0 = 0; j0 < TM; j0 += PJ) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const uint2 w = bw[i][g];
            const float b0 = unpack1_16<BF16>((uint16_t)(w.x & 0xFFFFu)), b1 = unpack1_16<BF16>((uint16_t)(w.x >> 16));
            const float b2 = unpack1_16<BF16>((uint16_t)(w.y & 0xFFFFu)), b3 = unpack1_16<BF16>((uint16_t)(w.y >> 16));
            uint8_t* const at = own + l32 * 256 + 16 * ((4 * i + g) ^ (l32 & 15)) + 8 * (h ^ (l32 >> 4));
#pragma unroll
            for (int j = j0; j < j0 + PJ; ++j) {
              uint2 o;
              o.x = pack2_16<BF16>(acc[i][j][4 * g] + b0, acc[i][j][4 * g + 1] + b1);
              o.y = pack2_16<BF16>(acc[i][j][4 * g + 2] + b2, acc[i][j][4 * g + 3] + b3);
              *reinterpret_cast<uint2*>(at + 32 * 256 * (j - j0)) = o;
            }
          }
        // eight reads in flight, then their stores: store x takes rows 4 x .. 4 x + 3, whose swizzle
        // depends on x % 4.  SEQ: written through the level-2 cache (sc0 sc1), so that one round's
        // outputs leave under the next one's products (16384 x 4608 x 1152: 93.5 against 98.2 us).
#pragma unroll
        for (int x0 = 0; x0 < 8 * PJ; x0 += 8) {
          v4i v[8];
#pragma unroll
          for (int y = 0; y < 8; ++y) v[y] = *reinterpret_cast<const v4i*>(from[y & 3] + 4096 * ((x0 + y) >> 2));
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const v4i w = y < 4 ? v[y] : v4i{v[y].z, v[y].w, v[y].x, v[y].y};
            __builtin_amdgcn_raw_buffer_store_b128(w, rY, (int)(to + 8u * N * (8 * j0 + x0 + y)), 0, SEQ ? 17 : 0);
          }
        }
      }
    } else {
      f8_gated_store<ACT, WIDE, TM>(acc, lds + C::TOP_OFF, wn, wrow_a, wrow_b, l32, h, m0, mleft, n0 >> 1, N, out, oscales);
    }
    if (!SEQ || (t += step) >= end) break;
    sbuf = (sbuf + (T + 15) / 16) & 1;
    lds_barrier();                             // the slot's reads are done, and all see the next stage 0
    if constexpr (!GATED) {
      at(t, m0, n0);
      bias_load(n0);
      uint32_t ko[2] = {k_off(128, 0), k_off(128, 1)};
      asm volatile("" : "+v"(ko[0]), "+v"(ko[1]));             // likewise
#pragma unroll
      for (int g = 0; g < NL; ++g) code_load(after, ko[g & 1], g);
    }
  }
}

using F8Large = F8Big<4, 2>;     // 256 x 256
using F8Half = F8Big<2, 3>;      // 256 x 128 tokens
using F8Low = F8Big<1, 3>;       // 256 x 64 tokens

// The first full_rows rows of 256-token tiles are whole tiles, grouped eight along M for reuse
// in the level-2 caches; the tokens below them are in tiles of 128, one for each of the last
// workgroups.  The others take whole tiles, one each or (SEQ) in turn.
template <int ACT, bool BF16, bool SEQ>
__global__ __launch_bounds__(256, 1) void f8_gemm_kernel(
    const uint8_t* __restrict__ wcodes, const uint8_t* __restrict__ wscales, const uint8_t* __restrict__ xcodes,
    const uint8_t* __restrict__ xscales, int64_t M, int N, int K, const uint16_t* __restrict__ bias,
    uint8_t* __restrict__ out, uint8_t* __restrict__ oscales, int full_rows) {
  __shared__ __align__(16) uint8_t lds[F8Large::LDS > F8Half::LDS ? F8Large::LDS : F8Half::LDS];
  const int tiles_n = ACT >= 0 ? (N + 127) / 128 : (N + 255) / 256;
  const int nfull = tiles_n * full_rows;
  const int rest = max(0, (int)((M + 127) / 128) - 2 * full_rows), nrest = tiles_n * rest;
  const int gfull = (int)gridDim.x - nrest;
  if ((int)blockIdx.x < gfull) {
    auto at = [&](int t, int64_t& m0, int& n0) {
      constexpr int GM = 8;
      const int pid = f8_remap(t, nfull);
      const int first = pid / (GM * tiles_n) * GM, rows = min(full_rows - first, GM), in = pid % (GM * tiles_n);
      m0 = 256LL * (first + in % rows);
      n0 = 256 * (in / rows);
    };
    f8_big_tiles<ACT, BF16, false, F8Large, SEQ>(lds, wcodes, wscales, xcodes, xscales, M, N, K, bias, out, oscales, at,
                                           blockIdx.x, nfull, gfull);
  } else {
    auto at = [&](int t, int64_t& m0, int& n0) {
      const int q = f8_remap(t, nrest);
      m0 = 256LL * full_rows + 128LL * (q % rest);
      n0 = 256 * (q / rest);
    };
    f8_big_tiles<ACT, BF16, false, F8Half, false>(lds, wcodes, wscales, xcodes, xscales, M, N, K, bias, out, oscales, at,
                                           (int)blockIdx.x - gfull, nrest, 1);
  }
}

template <bool BF16, bool WIDE, class C>
__global__ __launch_bounds__(256, 1) void f8_small_kernel(
    const uint8_t* __restrict__ wcodes, const uint8_t* __restrict__ wscales, const uint8_t* __restrict__ xcodes,
    const uint8_t* __restrict__ xscales, int64_t M, int N, int K, const uint16_t* __restrict__ bias,
    uint8_t* __restrict__ out) {
  __shared__ __align__(16) uint8_t lds[C::LDS];
  const int rows = (int)((M + C::BM - 1) / C::BM), pid = f8_remap(blockIdx.x, gridDim.x);
  f8_small_tile<BF16, WIDE, C>(lds, wcodes, wscales, xcodes, xscales, M, N, K, bias, out, (int64_t)C::BM * (pid % rows),
                         C::BN * (pid / rows));
}

// One tile per workgroup, grouped eight along M: 256 x 64 tokens for a gated call's middling token
// counts, 256 x 128 for all calls of more tokens whose products are to be in float32.
template <int ACT, bool BF16, bool WIDE, class C>
__global__ __launch_bounds__(256, 1) void f8_tiles_kernel(
    const uint8_t* __restrict__ wcodes, const uint8_t* __restrict__ wscales, const uint8_t* __restrict__ xcodes,
    const uint8_t* __restrict__ xscales, int64_t M, int N, int K, const uint16_t* __restrict__ bias,
    uint8_t* __restrict__ out, uint8_t* __restrict__ oscales) {
  __shared__ __align__(16) uint8_t lds[C::LDS];
  constexpr int GM = 8;
  const int tiles_n = ACT >= 0 ? (N + 127) / 128 : (N + 255) / 256, tiles_m = (int)((M + C::BM - 1) / C::BM);
  auto at = [&](int, int64_t& m0, int& n0) {
    const int pid = f8_remap(blockIdx.x, gridDim.x);
    const int first = pid / (GM * tiles_n) * GM, rows = min(tiles_m - first, GM), in = pid % (GM * tiles_n);
    m0 = (int64_t)C::BM * (first + in % rows);
    n0 = 256 * (in / rows);
  };
  f8_big_tiles<ACT, BF16, WIDE, C, false>(lds, wcodes, wscales, xcodes, xscales, M, N, K, bias, out, oscales, at, 0, 1,
                                          1);
}

template <int ACT, bool BF16, bool WIDE, class C>
static hipError_t tiles_launch(const uint8_t* xcodes, const uint8_t* xscales, int64_t M, int64_t K,
                               const uint8_t* wcodes, const uint8_t* wscales, int64_t N, const uint16_t* bias,
                               uint8_t* out, uint8_t* oscales, hipStream_t s) {
  const int64_t tiles_n = ACT >= 0 ? (N + 127) / 128 : (N + 255) / 256, tiles_m = (M + C::BM - 1) / C::BM;
  hipLaunchKernelGGL((f8_tiles_kernel<ACT, BF16, WIDE, C>), dim3((unsigned)(tiles_n * tiles_m)), dim3(256), 0, s, wcodes,
                     wscales, xcodes, xscales, M, (int)N, (int)K, bias, out, oscales);
  return hipGetLastError();
}

template <int ACT, bool BF16>
static hipError_t gemm_launch(const uint8_t* xcodes, const uint8_t* xscales, int64_t M, int64_t K,
                              const uint8_t* wcodes, const uint8_t* wscales, int64_t N, const uint16_t* bias,
                              uint8_t* out, uint8_t* oscales, hipStream_t s) {
  // A last round of tiles that leaves compute units idle costs nearly as much as a full one, so
  // the last rows of tiles may be split into tiles of 128 tokens, which take about 0.6 of a whole
  // one.  For each split: the fulls take their rounds, and the rest go to whichever compute units
  // are free first (those that had one full fewer, until the others come).  Measured (us) without
  // and with: gated 4096 x 11008 x 4096 (5.4 rounds) 306 and 298, linear 3000 x 8192 x 4096 (1.5) 89.5
  // and 84.9, 8192 x 4608 x 1152 (2.25) 53.7 and 52.9; tiles of 64 tokens gained at none of nine shapes.
  const int64_t tiles_n = ACT >= 0 ? (N + 127) / 128 : (N + 255) / 256, tiles_m = (M + 255) / 256;
  const int64_t cus = device_cu_count(), ntiles = tiles_n * tiles_m, rounds = (ntiles + cus - 1) / cus;
  int64_t full_rows = tiles_m;
  double best = (double)rounds - 0.02;       // a split has to gain
  for (int64_t rows = ntiles <= cus ? 0 : std::max<int64_t>(tiles_m - 4, 0); rows < tiles_m; ++rows) {
    const int64_t nfull = rows * tiles_n, nrest = tiles_n * ((M + 127) / 128 - 2 * rows);
    const int64_t late = nfull % cus;        // compute units with one full more
    double early_at = (double)(nfull / cus), late_at = early_at + 1.0, end = late ? late_at : early_at;
    for (int64_t left = nrest; left > 0;) {
      const bool l = late && late_at <= early_at;
      left -= l ? late : cus - late;
      end = std::max(end, (l ? late_at : early_at) += 0.6);
    }
    if (end < best) best = end, full_rows = rows;
  }
  // Several whole tiles in sequence on a workgroup, the next one's first loads under the present one's last
  // products: the more, the shorter their k.  Measured (us) without and with: linear 16384 x 6144 x 512
  // 83.6 and 77.2, 8192 x 8192 x 1024 80.3 and 76.7, 8192 x 4608 x 1152 54.6 and 52.3, 8192 x 4608 x 4096
  // 129.1 and 128.9, x 8192 244 and 244 (on another card 237 and 246), gated 4096 x 11008 x 2240 195 and 189.
  const int64_t nfull = full_rows * tiles_n, nrest = tiles_n * std::max<int64_t>((M + 127) / 128 - 2 * full_rows, 0);
  const bool seq = nfull > cus && K > 128 && K <= 4096;
  const dim3 blocks((unsigned)((seq ? cus : nfull) + nrest));
#define KQ_GEMM(SEQ)                                                                                                 \
  hipLaunchKernelGGL((f8_gemm_kernel<ACT, BF16, SEQ>), blocks, dim3(256), 0, s, wcodes, wscales, xcodes, xscales, M, \
                     (int)N, (int)K, bias, out, oscales, (int)full_rows)
  if (seq) KQ_GEMM(true);
  else KQ_GEMM(false);
#undef KQ_GEMM
  return hipGetLastError();
}

// The smallest tiles that give at most one workgroup per compute unit: fewer, larger tiles read
// less, but a chain of k over few compute units is bound by what one of them can take in.
template <bool BF16, bool WIDE>
static hipError_t linear_launch(const uint8_t* xcodes, const uint8_t* xscales, int64_t M, int64_t K,
                                const uint8_t* wcodes, const uint8_t* wscales, int64_t N, const uint16_t* bias,
                                uint8_t* Y, hipStream_t s) {
  if (rows_fit(M, (N + 31) / 32)) return rows_launch<-1, BF16>(WIDE, xcodes, xscales, M, K, wcodes, wscales, N, bias, Y, s);
  const int64_t cus = device_cu_count();
  auto tiles = [&](int64_t bn, int64_t bm) { return ((N + bn - 1) / bn) * ((M + bm - 1) / bm); };
#define KQ_TILE(...)                                                                                                \
  hipLaunchKernelGGL((f8_small_kernel<BF16, WIDE, F8Small<__VA_ARGS__>>),                                                  \
                     dim3((unsigned)tiles(F8Small<__VA_ARGS__>::BN, F8Small<__VA_ARGS__>::BM)), dim3(256), 0, s,     \
                     wcodes, wscales, xcodes, xscales, M, (int)N, (int)K, bias, Y)
  // measured (us) at 4096 x 4096 with 64 x 64 / 128 x 64 / 128 x 128 / 256 x 256: 200 tokens 12.0 /
  // 15.1 / 18.0 / 27.6, 512 tokens 18.4 / 16.4 / 18.9 / 29.0, 1024 tokens 33.6 / 30.6 / 22.5 / 30.5,
  // 2048 tokens 79 / 60 / 43 / 39; 512 tokens, 4096 x 1152 8.2 / 7.2 / 8.3 / 11.2
  if (tiles(64, 64) <= cus) KQ_TILE(1, 1, 8, 2);
  else if (tiles(128, 64) <= cus) KQ_TILE(2, 1, 4, 1);
  else if (tiles(128, 128) <= cus) KQ_TILE(2, 2, 4, 1);
  else if constexpr (WIDE) return tiles_launch<-1, BF16, true, F8Half>(xcodes, xscales, M, K, wcodes, wscales, N, bias, Y, nullptr, s);
  else return gemm_launch<-1, BF16>(xcodes, xscales, M, K, wcodes, wscales, N, bias, Y, nullptr, s);
#undef KQ_TILE
  return hipGetLastError();
}

hipError_t launch_f8_linear(bool bf16, bool precise, const uint8_t* xcodes, const uint8_t* xscales, int64_t M, int64_t K,
                            const uint8_t* wcodes, const uint8_t* wscales, int64_t N, const void* bias, void* Y,
                            hipStream_t s) {
  const auto go = bf16 ? precise ? linear_launch<true, true> : linear_launch<true, false>
                       : precise ? linear_launch<false, true> : linear_launch<false, false>;
  return go(xcodes, xscales, M, K, wcodes, wscales, N, static_cast<const uint16_t*>(bias), static_cast<uint8_t*>(Y), s);
}

size_t f8_gated_workspace_bytes(int64_t M, int64_t F, int64_t) { return gated_rows(M, F) ? (size_t)M * F * 4 : 0; }

template <int ACT, bool WIDE>
static hipError_t gated_launch(const uint8_t* xcodes, const uint8_t* xscales, int64_t M, int64_t K,
                               const uint8_t* wcodes, const uint8_t* wscales, int64_t F, uint8_t* codes,
                               uint8_t* scales, void* workspace, hipStream_t s) {
  if (gated_rows(M, F)) {
    // a workgroup's 16 columns are an eighth of a scale group: the outputs go through the
    // workspace in float32 and the quantizer
    const hipError_t e = rows_launch<ACT, false>(WIDE, xcodes, xscales, M, K, wcodes, wscales, F, nullptr, workspace, s);
    if (e != hipSuccess) return e;
    return launch_f8_quantize_f32(static_cast<const float*>(workspace), M, F, codes, scales, s);
  }
  // 64 tokens a tile while that is at most one workgroup per compute unit; measured (us) with 64 / 128
  // / 256 tokens: 128 tokens, 11008 x 4096 26.6 / 30.9 / 37; 203 tokens 45 / 30 / 37; 203 tokens, 5600 x
  // 2240 15.2 / 18.7 / 21
  const int64_t tiles = (F + 127) / 128 * ((M + F8Low::BM - 1) / F8Low::BM);
  if (tiles <= device_cu_count())
    return tiles_launch<ACT, false, WIDE, F8Low>(xcodes, xscales, M, K, wcodes, wscales, F, nullptr, codes, scales, s);
  if constexpr (WIDE)
    return tiles_launch<ACT, false, true, F8Half>(xcodes, xscales, M, K, wcodes, wscales, F, nullptr, codes, scales, s);
  else
    return gemm_launch<ACT, false>(xcodes, xscales, M, K, wcodes, wscales, F, nullptr, codes, scales, s);
}

hipError_t launch_f8_gated(int act, bool precise, const uint8_t* xcodes, const uint8_t* xscales, int64_t M, int64_t K,
                           const uint8_t* wcodes, const uint8_t* wscales, int64_t F, uint8_t* codes, uint8_t* scales,
                           void* workspace, hipStream_t s) {
  const auto go = act == 0   ? precise ? gated_launch<0, true> : gated_launch<0, false>
                  : act == 1 ? precise ? gated_launch<1, true> : gated_launch<1, false>
                             : precise ? gated_launch<2, true> : gated_launch<2, false>;
  return go(xcodes, xscales, M, K, wcodes, wscales, F, codes, scales, workspace, s);
}

}  // namespace kq
