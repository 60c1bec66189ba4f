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
// GELU's g Phi(g) goes through erfc for the same reason.  The exponential is the hardware's
// exp2 and the quotient its reciprocal (each good to one step): the correctly rounded forms
// cost five times as many instructions, and the result is rounded to four bits next.
template <int ACT>
__device__ __forceinline__ float f8_act(float g) {
  if (ACT == 1) return 0.5f * g * erfcf(-0.70710678118654752f * g);
  constexpr float L = 1.4426950408889634f;              // log2 e
  const float x = ACT == 0 ? -L * g : -1.5957691216057308f * L * fmaf(0.044715f * g * g, g, g);
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x));
}

// ---------------------------------------------------------------------------------
// Few tokens (up to 16 MT): the weights' bytes bound it.  A workgroup takes 16 weight rows
// (gated: 16 gate rows and the 16 up rows of the same columns) and all tokens; its NW
// wavefronts take the 128-wide groups of k in turn, U groups of loads in flight each, and
// their sums are added through LDS in wavefront order.  The codes are widened to bf16 with
// their scale applied (exact: four significant bits) and multiplied by the bf16 matrix
// instruction, which sums in float32: there is time for it under the loads, and it does not
// drop bits as the 8-bit instruction does.  Lane l holds row l % 16 and, of each group, bytes
// 16 (l / 16) .. + 15 of both 64-byte halves, the same for both operands.
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));

// Eight of the sixteen codes in a piece (p = 0, 1), widened and scaled.
template <int P>
__device__ __forceinline__ v8b f8_widen8(const v4i& w, float scale) {
  const uint32_t lo = (uint32_t)w[2 * P], hi = (uint32_t)w[2 * P + 1];
  const v2b a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const v2b b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const v2b c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const v2b d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return v8b{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

template <int ACT, bool BF16, int MT, int NW, int U>   // ACT -1: the linear
__global__ __launch_bounds__(64 * NW) void f8_rows_kernel(const uint8_t* __restrict__ wcodes,
                                                          const uint8_t* __restrict__ wscales,
                                                          const uint8_t* __restrict__ xcodes,
                                                          const uint8_t* __restrict__ xscales, int M, int N, int K,
                                                          const uint16_t* __restrict__ bias, void* __restrict__ out) {
  constexpr int RT = ACT >= 0 ? 2 : 1;
  __shared__ v4f part[NW][RT * MT][64];
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int SC = (int)f8_scale_cols(K), T = (K + 127) / 128;
  const int n0 = 16 * blockIdx.x;
  __amdgpu_buffer_rsrc_t rw[RT], rws[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    rw[i] = make_rsrc(wcodes + (int64_t)(n0 + i * N) * K, 16LL * K);
    rws[i] = make_rsrc(wscales + (int64_t)(n0 + i * N) * SC, 16LL * SC);
  }
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(xcodes, (int64_t)M * K), rxs = make_rsrc(xscales, (int64_t)M * SC);
  v4f acc[RT][MT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  for (int t0 = wid; t0 < T; t0 += NW * U) {
    v4i w[U][RT][2], x[U][MT][2];
    uint32_t ws[U][RT], xs[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * NW;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int k = 128 * t + 64 * p + 16 * q;
        const bool live = k < K;                               // K is a multiple of 16
#pragma unroll
        for (int i = 0; i < RT; ++i)
          w[u][i][p] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rw[i], live ? r * K + k : KQ_OOB, 0, 0));
#pragma unroll
        for (int j = 0; j < MT; ++j)
          x[u][j][p] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rx, live ? (16 * j + r) * K + k : KQ_OOB, 0, 0));
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) ws[u][i] = __builtin_amdgcn_raw_buffer_load_b8(rws[i], t < T ? r * SC + t : KQ_OOB, 0, 0);
#pragma unroll
      for (int j = 0; j < MT; ++j) xs[u][j] = __builtin_amdgcn_raw_buffer_load_b8(rxs, t < T ? (16 * j + r) * SC + t : KQ_OOB, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);                         // all loads out before the first product
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v8b wb[RT][4];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const float s = __uint_as_float(ws[u][i] << 23);
        wb[i][0] = f8_widen8<0>(w[u][i][0], s);
        wb[i][1] = f8_widen8<1>(w[u][i][0], s);
        wb[i][2] = f8_widen8<0>(w[u][i][1], s);
        wb[i][3] = f8_widen8<1>(w[u][i][1], s);
      }
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const float s = __uint_as_float(xs[u][j] << 23);
        const v8b xb[4] = {f8_widen8<0>(x[u][j][0], s), f8_widen8<1>(x[u][j][0], s), f8_widen8<0>(x[u][j][1], s),
                           f8_widen8<1>(x[u][j][1], s)};
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < RT; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[i][c], xb[c], acc[i][j], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) part[wid][i * MT + j][lane] = acc[i][j];
  __syncthreads();
  // wavefront j sums and stores tokens 16 j .. + 15: lane l holds columns 4 (l / 16) .. + 3 of token l % 16
  for (int j = wid; j < MT; j += NW) {
    v4f s[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      s[i] = part[0][i * MT + j][lane];
#pragma unroll
      for (int v = 1; v < NW; ++v) s[i] += part[v][i * MT + j][lane];
    }
    const int m = 16 * j + r, col = n0 + 4 * q;
    if (m >= M) continue;
    if constexpr (ACT >= 0) {
      v4f y;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = f8_act<ACT>(s[0][e]) * s[RT - 1][e];
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

template <int ACT, bool BF16>
static hipError_t rows_launch(const uint8_t* xcodes, const uint8_t* xscales, int64_t M, int64_t K,
                              const uint8_t* wcodes, const uint8_t* wscales, int64_t N, const uint16_t* bias,
                              void* out, hipStream_t s) {
  const dim3 g((unsigned)(N / 16));
#define KQ_ROWS(MT, NW, U)                                                                                          \
  hipLaunchKernelGGL((f8_rows_kernel<ACT, BF16, MT, NW, U>), g, dim3(64 * NW), 0, s, wcodes, wscales, xcodes, xscales, \
                     (int)M, (int)N, (int)K, bias, out)
  if (M <= 16) {
    if (K <= 4096) KQ_ROWS(1, 8, 4);
    else KQ_ROWS(1, 16, 4);
  } else if (M <= 32) {
    KQ_ROWS(2, 8, 2);
  } else {
    KQ_ROWS(4, 8, 2);
  }
#undef KQ_ROWS
  return hipGetLastError();
}

// ---------------------------------------------------------------------------------
// Many tokens: tiles of 256 weight rows by 64 TM token rows on four wavefronts (2 x 2), each
// 128 x 32 TM as 4 x TM blocks of 32 x 32 (TM = 4: 256 float32 accumulators a lane).  The
// operands go from global memory straight into LDS, 64 k (one matrix instruction) a stage,
// four stages deep; a stage's row is four 16-byte chunks, XOR-swizzled so that the fragment
// reads (16 rows x one chunk) and the staging writes hit distinct banks.  Lane l of half
// h = l / 32 takes chunks h and 2 + h of its row as its 32 values of k.
// Per stage: wait for the next stage's loads, one barrier, then 4 TM products of 64 cycles
// with the next stage's fragment reads and the loads of the stage after the ring spread
// between them (the barrier has freed this stage's own slot: its fragments are in registers).
// Scale bytes come 16 at a time for each row (2048 k, so seldom) into a double-buffered area.
struct F8Tile {
  static constexpr int NS = 4;                                 // stages
  static constexpr int A_BYTES = 256 * 64;
  static constexpr int STAGE = 2 * A_BYTES;
  static constexpr int SC_OFF = NS * STAGE;                    // two scale groups: 256 + 256 rows x 16 bytes
  static constexpr int SC_BYTES = 512 * 16;
  static constexpr int BIAS_OFF = SC_OFF + 2 * SC_BYTES;       // 64 lanes x 16 bytes (256 biases used)
  static constexpr int TOP_OFF = BIAS_OFF + 1024;              // gated: 2 x 256 maxima
  static constexpr int LDS = TOP_OFF + 2048;                   // 150528 bytes
};

__device__ __forceinline__ int f8_swz(int row) { return ((row >> 1) ^ (row >> 2)) & 3; }

// ACT -1: the linear, weight rows n0 .. n0 + 255.  Gated: rows f0 .. f0 + 127 of both halves,
// f0 = n0 / 2; wavefront column wn holds gate and up of columns f0 + 64 wn .. + 63, so that a
// lane has both factors of an output, and the tile's 128 columns are one scale group.
template <int ACT, bool BF16, int TM>
__device__ __forceinline__ void f8_tile(uint8_t* __restrict__ lds, const uint8_t* __restrict__ wcodes,
                                        const uint8_t* __restrict__ wscales, const uint8_t* __restrict__ xcodes,
                                        const uint8_t* __restrict__ xscales, int64_t M, int N, int K,
                                        const uint16_t* __restrict__ bias, uint8_t* __restrict__ out,
                                        uint8_t* __restrict__ oscales, int64_t m0, int n0) {
  using C = F8Tile;
  constexpr bool GATED = ACT >= 0;
  constexpr int NS = C::NS, NL = 4 + TM, NM = 4 * TM, NR = 2 * (4 + TM);
  // the thread index, hidden from the compiler, so that it does not keep every lane-dependent
  // offset live across a tile loop
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wid & 1, wm = wid >> 1;
  const int l32 = lane & 31, h = lane >> 5;
  const int SC = (int)f8_scale_cols(K);
  const int nk = 2 * ((K + 127) / 128);                        // stages: whole groups, zeros past K

  // wave w stages weight rows 64 w .. 64 w + 63 of the tile and token rows 16 TM w .. + 16 TM - 1
  const int64_t arow = GATED ? (int64_t)(wid & 1) * N + (n0 >> 1) + 64 * (wid >> 1) : (int64_t)n0 + 64 * wid;
  const int64_t aleft = GATED ? N - (n0 >> 1) - 64 * (wid >> 1) : N - n0 - 64 * wid;
  const v4i rA = rsrc_words(wcodes + arow * K, aleft * K);
  const v4i rAS = rsrc_words(wscales + arow * SC, aleft * SC);
  const v4i rB = rsrc_words(xcodes + m0 * K, (M - m0) * K);
  const v4i rBS = rsrc_words(xscales + m0 * SC, (M - m0) * SC);

  const uint32_t lds0 = lds_addr(lds);
  const int csw = 16 * ((lane & 3) ^ f8_swz(lane >> 2));
  // unsigned: an offset past the end is KQ_OOB plus at most 2^28 and stays past every range
  const uint32_t ogA = (lane >> 2) * K + csw, ogB = (16 * TM * wid + (lane >> 2)) * K + csw;
  auto k_off = [&](int ks) -> uint32_t { return 64 * ks + csw < K ? 64 * ks : KQ_OOB; };
  auto code_load = [&](int ks, uint32_t ko, int g) {                // load g (0 .. NL - 1) of stage ks
    const uint32_t st = lds0 + (uint32_t)((ks % NS) * C::STAGE);
    if (g < 4) lds_load16(rA, st + (64 * wid + 16 * g) * 64, (int)(ogA + 16 * g * K + ko));
    else lds_load16(rB, st + C::A_BYTES + (16 * TM * wid + 16 * (g - 4)) * 64, (int)(ogB + 16 * (g - 4) * K + ko));
  };
  // scale bytes of stages 32 grp .. 32 grp + 31, issued only when skip is zero: the branch is
  // inside the assembly so that the loop body stays one block for the scheduler.  A row's last
  // piece may run into the next row; those bytes are never read.
  const uint32_t osc = lane * SC, oscb = wid < TM ? (64 * wid + lane) * SC : KQ_OOB;
  auto scale_loads = [&](int grp, int skip) {
    const uint32_t sc = lds0 + (uint32_t)(C::SC_OFF + (grp & 1) * C::SC_BYTES + 16 * 64 * wid);
    const uint32_t ko = 32 * grp < nk ? 16 * grp : KQ_OOB;
    asm volatile(
        "s_cmp_lg_u32 %0, 0\n\t"
        "s_cbranch_scc1 1f\n\t"
        "s_mov_b32 m0, %1\n\t"
        "buffer_load_dwordx4 %3, %5, 0 offen lds\n\t"
        "s_mov_b32 m0, %2\n\t"
        "buffer_load_dwordx4 %4, %6, 0 offen lds\n"
        "1:"
        :: "s"(__builtin_amdgcn_readfirstlane(skip)), "s"(__builtin_amdgcn_readfirstlane(sc)),
           "s"(__builtin_amdgcn_readfirstlane(sc + 256 * 16)), "v"(osc + ko), "v"(oscb + (wid < TM ? ko : 0)),
           "s"(rAS), "s"(rBS)
        : "memory", "m0", "scc");
  };

  const int wrow_a = 128 * wn, wrow_b = 32 * TM * wm;
  const int sw = f8_swz(l32);                                  // the same for every block of 32 rows
  const int fa = (wrow_a + l32) * 64, fb = C::A_BYTES + (wrow_b + l32) * 64;
  const int c0 = 16 * (h ^ sw), c1 = 16 * ((2 + h) ^ sw);
  auto read_half = [&](const uint8_t* st, int q, v8i* a, v8i* b) {   // half fragment q (0 .. NR - 1)
    const int f = q >> 1;
    const int at = (f < 4 ? fa + 2048 * f : fb + 2048 * (f - 4)) + ((q & 1) ? c1 : c0);
    const v4i v = *reinterpret_cast<const v4i*>(st + at);
    v8i& d = f < 4 ? a[f] : b[f - 4];
#pragma unroll
    for (int e = 0; e < 4; ++e) d[4 * (q & 1) + e] = v[e];
  };
  const int sa_at = 16 * (wrow_a + l32), sb_at = 256 * 16 + 16 * (wrow_b + l32);
  auto read_scale = [&](int ks, int q) -> int {                // scale of fragment q for the pair of stages from ks
    const uint8_t* sc = lds + C::SC_OFF + ((ks >> 5) & 1) * C::SC_BYTES + ((ks >> 1) & 15);
    return sc[q < 4 ? sa_at + 512 * q : sb_at + 512 * (q - 4)];
  };

  v16f acc[4][TM];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  if (!GATED && wid == 0) {                                    // without a bias, or past N: zeros
    const v4i rW = rsrc_words(bias + n0, bias ? (int64_t)(N - n0) * 2 : 0);
    lds_load16(rW, lds0 + C::BIAS_OFF, lane < 32 ? 16 * lane : KQ_OOB);
  }
  scale_loads(0, 0);
#pragma unroll
  for (int p = 0; p < NS; ++p)
#pragma unroll
    for (int g = 0; g < NL; ++g) code_load(p, k_off(p), g);
  __builtin_amdgcn_s_waitcnt(waitcnt_vm((NS - 1) * NL));       // biases, scales and stage 0
  lds_barrier();
  v8i a[2][4], b[2][TM];
  int s[4 + TM];
#pragma unroll
  for (int q = 0; q < 4 + TM; ++q) s[q] = read_scale(0, q);
#pragma unroll
  for (int q = 0; q < NR; ++q) read_half(lds, q, a[0], b[0]);

  for (int ks = 0; ks < nk; ks += 2) {
    int ns[4 + TM];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // stage ks + u + 1 has landed once at most those of the two stages behind it are outstanding
      __builtin_amdgcn_s_waitcnt(waitcnt_vm((NS - 2) * NL));
      lds_barrier();
      if (u == 0) scale_loads((ks >> 5) + 1, ks & 31);
      const uint8_t* const nxt = lds + ((ks + u + 1) % NS) * C::STAGE;
      const uint32_t ko = k_off(ks + u + NS);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        const int i = m / TM, j = m % TM;
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a[u][i], b[u][j], acc[i][j], 0, 0, 0, s[i], 0, s[4 + j]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = NR * m / NM; q < NR * (m + 1) / NM; ++q) read_half(nxt, q, a[1 - u], b[1 - u]);
        if (u == 1) {
#pragma unroll
          for (int q = (4 + TM) * m / NM; q < (4 + TM) * (m + 1) / NM; ++q) ns[q] = read_scale(ks + 2, q);
        }
#pragma unroll
        for (int g = NL * m / NM; g < NL * (m + 1) / NM; ++g) code_load(ks + u + NS, ko, g);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int q = 0; q < 4 + TM; ++q) s[q] = ns[q];
  }
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));                   // no load may land in LDS after this tile

  if constexpr (!GATED) {
    const __amdgpu_buffer_rsrc_t rY = make_rsrc(out + m0 * N * 2, (M - m0) * N * 2);
    const uint32_t* const bias_t = reinterpret_cast<const uint32_t*>(lds + C::BIAS_OFF);
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int ml = wrow_b + 32 * j + l32;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
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
  } else {
    // outputs in place of the gates, the maximum of each token's 64 columns to LDS, and after
    // the barrier the scale of its 128 (rows past F are zeros on both sides and stay zeros)
    uint32_t* const tops = reinterpret_cast<uint32_t*>(lds + C::TOP_OFF);
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float v = f8_act<ACT>(acc[i][j][e]) * acc[i + 2][j][e];
          acc[i][j][e] = v;
          top = umax32(top, abs_bits(v));
        }
      top = umax32(top, (uint32_t)__shfl_xor((int)top, 32, 64));
      if (h == 0) tops[256 * wn + wrow_b + 32 * j + l32] = top;
    }
    lds_barrier();
    const int f0 = n0 >> 1, OS = (int)f8_scale_cols(N), grp = f0 >> 7;
    const __amdgpu_buffer_rsrc_t rQ = make_rsrc(out + m0 * N, (M - m0) * N);
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int ml = wrow_b + 32 * j + l32;
      const uint32_t byte = f8_scale_byte(umax32(tops[ml], tops[256 + ml]));
      const bool bad = byte == 255u;
      const float inv = bad ? 1.0f : f8_inv_scale(byte);
      if (wn == 0 && h == 0 && m0 + ml < M) {
        uint8_t* const row = oscales + (m0 + ml) * OS;
        row[grp] = (uint8_t)byte;
        if (f0 + 128 >= N)
          for (int q = grp + 1; q < OS; ++q) row[q] = 0;       // padding
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
        const int col = f0 + 64 * wn + 32 * i + 16 * h;
        __builtin_amdgcn_raw_buffer_store_b128(outv, rQ, col < N ? ml * N + col : KQ_OOB, 0, 0);
      }
    }
  }
}

// The first full_rows rows of 256-token tiles are whole tiles, grouped eight along M for reuse
// in the level-2 caches; the rows below them are tiles of 128 tokens.  Each workgroup loops over
// every grid-th tile.  Consecutive tile numbers, which the dispatcher deals out to the compute
// dies in turn, are remapped so that each die holds a contiguous run of tiles.
template <int ACT, bool BF16>
__global__ __launch_bounds__(256, 1) void f8_gemm_kernel(
    const uint8_t* __restrict__ wcodes, const uint8_t* __restrict__ wscales, const uint8_t* __restrict__ xcodes,
    const uint8_t* __restrict__ xscales, int64_t M, int N, int K, const uint16_t* __restrict__ bias,
    uint8_t* __restrict__ out, uint8_t* __restrict__ oscales, int full_rows) {
  __shared__ __align__(16) uint8_t lds[F8Tile::LDS];
  const int tiles_n = ACT >= 0 ? (N + 127) / 128 : (N + 255) / 256;
  const int nfull = tiles_n * full_rows;
  const int hrows = max(0, (int)((M + 127) / 128) - 2 * full_rows), nhalf = tiles_n * hrows;
  auto remap = [](int pid, int n) {
    const int per = n / 8;
    return pid < 8 * per ? (pid % 8) * per + pid / 8 : pid;
  };
  for (int t = blockIdx.x; t < nfull + nhalf; t += gridDim.x) {
    if (t < nfull) {
      constexpr int GM = 8;
      const int pid = remap(t, nfull);
      const int first = pid / (GM * tiles_n) * GM, rows = min(full_rows - first, GM), in = pid % (GM * tiles_n);
      f8_tile<ACT, BF16, 4>(lds, wcodes, wscales, xcodes, xscales, M, N, K, bias, out, oscales,
                            256LL * (first + in % rows), 256 * (in / rows));
    } else {
      const int q = remap(t - nfull, nhalf);
      f8_tile<ACT, BF16, 2>(lds, wcodes, wscales, xcodes, xscales, M, N, K, bias, out, oscales,
                            256LL * full_rows + 128LL * (q % hrows), 256 * (q / hrows));
    }
    __syncthreads();                         // the next tile's loads stay off what this one's epilogue reads
  }
}

template <int ACT, bool BF16>
static hipError_t gemm_launch(const uint8_t* xcodes, const uint8_t* xscales, int64_t M, int64_t K,
                              const uint8_t* wcodes, const uint8_t* wscales, int64_t N, const uint16_t* bias,
                              uint8_t* out, uint8_t* oscales, hipStream_t s) {
  // A last round of tiles that leaves compute units idle costs nearly as much as a full one:
  // its tile rows go to tiles of 128 tokens when those fit in one round; otherwise the rounds
  // are made even, each workgroup (a multiple of the 8 dies) taking every grid-th tile.
  const int64_t tiles_n = ACT >= 0 ? (N + 127) / 128 : (N + 255) / 256, tiles_m = (M + 255) / 256;
  const int64_t cus = device_cu_count(), ntiles = tiles_n * tiles_m, tail = ntiles % cus;
  int64_t full_rows = tiles_m;
  if (tail > 0) {
    const int64_t hr = (tail + tiles_n - 1) / tiles_n;
    if (tiles_n * ((M + 127) / 128 - 2 * (tiles_m - hr)) <= cus) full_rows = tiles_m - hr;
  }
  int64_t grid = tiles_n * full_rows;
  if (full_rows == tiles_m) {
    const int64_t rounds = (ntiles + cus - 1) / cus;
    grid = std::min(grid, ((ntiles + rounds - 1) / rounds + 7) / 8 * 8);
  } else {
    grid += tiles_n * ((M + 127) / 128 - 2 * full_rows);
  }
  hipLaunchKernelGGL((f8_gemm_kernel<ACT, BF16>), dim3((unsigned)grid), dim3(256), 0, s, wcodes, wscales, xcodes,
                     xscales, M, (int)N, (int)K, bias, out, oscales, (int)full_rows);
  return hipGetLastError();
}

size_t f8_linear_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

template <bool BF16>
static hipError_t linear_launch(const uint8_t* xcodes, const uint8_t* xscales, int64_t M, int64_t K,
                                const uint8_t* wcodes, const uint8_t* wscales, int64_t N, const uint16_t* bias,
                                uint8_t* Y, hipStream_t s) {
  if (M > 64) return gemm_launch<-1, BF16>(xcodes, xscales, M, K, wcodes, wscales, N, bias, Y, nullptr, s);
  return rows_launch<-1, BF16>(xcodes, xscales, M, K, wcodes, wscales, N, bias, Y, s);
}

hipError_t launch_f8_linear(bool bf16, const uint8_t* xcodes, const uint8_t* xscales, int64_t M, int64_t K,
                            const uint8_t* wcodes, const uint8_t* wscales, int64_t N, const void* bias, void* Y,
                            void* workspace, hipStream_t s) {
  const uint16_t* b = static_cast<const uint16_t*>(bias);
  uint8_t* y = static_cast<uint8_t*>(Y);
  return bf16 ? linear_launch<true>(xcodes, xscales, M, K, wcodes, wscales, N, b, y, s)
              : linear_launch<false>(xcodes, xscales, M, K, wcodes, wscales, N, b, y, s);
}

size_t f8_gated_workspace_bytes(int64_t M, int64_t F, int64_t) { return M > 64 ? 0 : (size_t)M * F * 4; }

template <int ACT>
static hipError_t gated_launch(const uint8_t* xcodes, const uint8_t* xscales, int64_t M, int64_t K,
                               const uint8_t* wcodes, const uint8_t* wscales, int64_t F, uint8_t* codes,
                               uint8_t* scales, void* workspace, hipStream_t s) {
  if (M > 64) return gemm_launch<ACT, false>(xcodes, xscales, M, K, wcodes, wscales, F, nullptr, codes, scales, s);
  const hipError_t e = rows_launch<ACT, false>(xcodes, xscales, M, K, wcodes, wscales, F, nullptr, workspace, s);
  if (e != hipSuccess) return e;
  return launch_f8_quantize_f32(static_cast<const float*>(workspace), M, F, codes, scales, s);
}

hipError_t launch_f8_gated(int act, const uint8_t* xcodes, const uint8_t* xscales, int64_t M, int64_t K,
                           const uint8_t* wcodes, const uint8_t* wscales, int64_t F, uint8_t* codes, uint8_t* scales,
                           void* workspace, hipStream_t s) {
  switch (act) {
    case 0: return gated_launch<0>(xcodes, xscales, M, K, wcodes, wscales, F, codes, scales, workspace, s);
    case 1: return gated_launch<1>(xcodes, xscales, M, K, wcodes, wscales, F, codes, scales, workspace, s);
    default: return gated_launch<2>(xcodes, xscales, M, K, wcodes, wscales, F, codes, scales, workspace, s);
  }
}

}  // namespace kq
