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

// 64 x 64 output tile, 2 x 2 wavefronts of 32 x 32, operands straight from global memory.
template <int ACT, bool BF16>   // ACT -1: the linear
__global__ __launch_bounds__(256) void f8_simple_kernel(const uint8_t* __restrict__ wcodes,
                                                        const uint8_t* __restrict__ wscales,
                                                        const uint8_t* __restrict__ xcodes,
                                                        const uint8_t* __restrict__ xscales, int64_t M, int N, int K,
                                                        const uint16_t* __restrict__ bias, void* __restrict__ out) {
  constexpr bool GATED = ACT >= 0;
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
      static_cast<float*>(out)[m * N + col] = f8_act<ACT>(v) * acc[GATED ? 1 : 0][q];
    } else {
      if (bias) v += unpack1_16<BF16>(bias[col]);
      static_cast<uint16_t*>(out)[m * N + col] = (uint16_t)pack2_16<BF16>(v, 0.0f);
    }
  }
}

static dim3 simple_grid(int64_t M, int64_t N) { return dim3((unsigned)((N + 63) / 64), (unsigned)((M + 63) / 64)); }

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
  hipLaunchKernelGGL((f8_simple_kernel<-1, BF16>), simple_grid(M, N), dim3(256), 0, s, wcodes, wscales, xcodes,
                     xscales, M, (int)N, (int)K, bias, Y);
  return hipGetLastError();
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
  hipLaunchKernelGGL((f8_simple_kernel<ACT, false>), simple_grid(M, F), dim3(256), 0, s, wcodes, wscales, xcodes,
                     xscales, M, (int)F, (int)K, nullptr, workspace);
  const hipError_t e = hipGetLastError();
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
