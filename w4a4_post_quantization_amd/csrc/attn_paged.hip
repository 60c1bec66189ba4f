// Attention of one new token a sequence over pages of cached keys and values, and the pages' filling.
//
// The cache's bytes bound it.  The batch's keys are cut into blocks of 64 (a key head's blocks after one
// another, then the next head's, then the next sequence's) and the blocks are dealt to a fixed number of
// workgroups in equal runs, whatever the lengths: a run may end inside a head's keys and begin inside
// another's.  The part of a run in one head is a piece.  Pieces that are whole heads go out at once; of a head
// that several runs share, each leaves its unnormalized sum, maximum and sum of weights in the
// workspace (a run has two such at most), and a second kernel joins them in a fixed order.
//
// Within a run, each of two wavefronts takes 32 keys of a block, through a ring of two slots of its own in
// LDS: the next block's loads (the next piece's first ones, too) are in flight while the present one is
// multiplied, and the loop has no barrier.  As for prompts everything is transposed:
// S^T = K Q^T with the key head's queries as 16 columns, O^T += V^T P^T in the order of keys in which the
// scores came out, V^T by transposing reads.  8-bit rows are widened exactly; their scales go to the scores
// (keys) and to the weights (values).  The weights are multiplied as sums of 16-bit numbers, three of bf16 or
// two of fp16, as exactly as float32 holds them; there is time for the products (one number less: 0 to 0.4 us less a call,
// but codes further from 64 bits than float32's own, 1 to 2e-4 of the norm and 0.2 to 1e-4).
//
// Measured with 32 / 8 heads of 128: 160 sequences of 200 to 8000 in 8 bits (1.28 GB) 241 us, 5.3 TB/s (a copy reaches 5.1);
// two of 131072 in 8 bits 103 us, 5.2 TB/s; 37 of 50 to 4000 in 16 bits from HBM 56 us, 4.7 TB/s; joins 4 to 7 us.
#include "kq_attn.hpp"
#include "kq_launch.hpp"

namespace kq {

namespace {

// Lengths are held to what the table's rows can hold.
__device__ __forceinline__ int held(const Pages& c, int32_t len) {
  return (int)min((int64_t)max(len, 0), (int64_t)c.width * c.page);
}
// Blocks of a sequence: 32 keys for each of a workgroup's NW wavefronts.
template <int NW>
__device__ __forceinline__ int blocks_in(int len) { return (int)(((int64_t)len + 32 * NW - 1) / (32 * NW)); }

// An entry at an index that the whole wavefront shares, as a scalar load: a vector load would have to be
// waited for together with the rings'.
__device__ __forceinline__ int32_t scalar_at(const int32_t* p, int64_t i) {
  return ((const __attribute__((address_space(4))) int32_t*)p)[i];
}
__device__ __forceinline__ int length_of(const Pages& c, int b) { return held(c, scalar_at(c.lengths, b)); }

// Sums over the lanes up to each one.  Of blocks: B width page <= 2^37 and B <= 2^20, so all sequences together have up to
// 2^31 + 2^20, which 32 bits hold without a sign.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  const int lane = threadIdx.x & 63;
  // within rows of 16 by shifts, then the rows' totals
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false);      // row_shr:1
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false);
  const uint32_t t0 = __builtin_amdgcn_readlane(v, 15), t1 = __builtin_amdgcn_readlane(v, 31), t2 = __builtin_amdgcn_readlane(v, 47);
  return v + (lane >= 16 ? t0 : 0) + (lane >= 32 ? t1 : 0) + (lane >= 48 ? t2 : 0);
}

// Block x of N belongs to run ((x + 1) W - 1) / N.
__device__ __forceinline__ int64_t run_start(int64_t w, int64_t N, int W) { return w * N / W; }

// A piece: blocks j0 .. j1 - 1 of the nb of one unit (a key head, or 16 of its queries where there are more) of
// sequence b, of len keys.
struct Piece {
  int b, unit, j0, j1, nb, len;
};

// What the joining kernel has to know of a run: its first piece, and the blocks of the whole batch.
struct Run {
  int64_t N;
  int32_t b, unit, j0, nb, pad[2];
};

// The run's first piece and its number of blocks (0: none); N and W (no run is to be empty) for all runs.
template <int NW>
__device__ int64_t find_run(const Pages& c, int HH, int w, int& W, int64_t& N, Piece& p) {
  const int lane = threadIdx.x & 63;
  auto length = [&](int b) { return b < c.B ? held(c, c.lengths[b]) : 0; };
  // up to 64 sequences: the scan that the search needs has the sum, too
  const int len0 = length(lane);
  const uint32_t upto0 = wave_scan(blocks_in<NW>(len0));
  uint32_t all = __builtin_amdgcn_readlane(upto0, 63);
  if (c.B > 64) {
    uint32_t more = 0;
    for (int b = 64; b < c.B; b += 64) more += blocks_in<NW>(length(b + lane));
    all += (uint32_t)__builtin_amdgcn_readlane(wave_scan(more), 63);
  }
  N = (int64_t)all * HH;
  W = (int)min((int64_t)W, N);
  if (w >= W) return 0;
  const int64_t x = run_start(w, N, W);
  const uint32_t y = (uint32_t)(x / HH);                     // the block, counting one unit of each sequence
  uint32_t base = 0;
  for (int b0 = 0; b0 < c.B; b0 += 64) {
    const int len = b0 == 0 ? len0 : length(b0 + lane);
    const uint32_t upto = b0 == 0 ? upto0 : wave_scan(blocks_in<NW>(len));
    const uint64_t hit = __ballot(y < base + upto);
    if (hit) {
      const int i = __builtin_ctzll(hit);
      p.b = b0 + i;
      p.len = __builtin_amdgcn_readlane(len, i);
      p.nb = blocks_in<NW>(p.len);
      const int64_t in = x - (int64_t)(base + (uint32_t)__builtin_amdgcn_readlane(upto, i) - (uint32_t)p.nb) * HH;
      p.unit = (int)(in / p.nb);
      p.j0 = (int)(in % p.nb);
      const int64_t blocks = run_start(w + 1, N, W) - x;
      p.j1 = (int)min((int64_t)p.nb, p.j0 + blocks);
      return blocks;
    }
    base += (uint32_t)__builtin_amdgcn_readlane(upto, 63);
  }
  return 0;
}

__device__ __forceinline__ float row_pair_max(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float row_pair_sum(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// 16 bytes from each active lane's own address into LDS at lds + 16 x lane.
__device__ __forceinline__ void lds_load16_at(uint32_t lds, const void* p) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, off"
               :: "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(p) : "memory", "m0");
}

// 2^(byte - 127); 0 stands for 2^-127, which is no normal float, and 255 for NaN.
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}

// The scales of sixteen bytes.  Where none is 0 or 255 a shift and a mask do (the tests of each byte cost a call of one
// short sequence 0.3 us).
__device__ __forceinline__ void e8m0_values(const uint32_t (&w)[4], float (&f)[16]) {
  float lo = INFINITY, hi = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int at = 8 * (i & 3);
    f[i] = __uint_as_float((at < 24 ? w[i >> 2] << (23 - at) : w[i >> 2] >> 1) & 0x7F800000u);
    lo = fminf(lo, f[i]), hi = fmaxf(hi, f[i]);
  }
  if (__builtin_expect(__any(!(lo > 0.0f && hi < INFINITY)), 0)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = e8m0_value((w[i >> 2] >> (8 * (i & 3))) & 255u);
  }
}

// Eight E4M3 codes as 16-bit values (exact).
template <bool BF16>
__device__ __forceinline__ v4u widen8(uint32_t lo, uint32_t hi) {
  v4u r;
  if constexpr (BF16) {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true));
  } else {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true));
  }
  return r;
}

// One row's eight values d = 8 i .. + 7 (i = lane % 16, the row's 16 lanes hold it all) into the output.
template <bool BF16>
__device__ __forceinline__ void store_row(const float* o, const PagedArgs& a, int b, int head, int i) {
  const int D = a.c.D;
  const int64_t row = (int64_t)b * a.Hq + head;
  if (a.scales) {                                            // D is 128
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = umax32(top, abs_bits(o[e]));
    const uint32_t byte = f8_scale_byte(row16_umax(top));
    const bool bad = byte == 255u;
    const float inv = bad ? 1.0f : f8_inv_scale(byte);
    const uint2 w = {bad ? 0x7F7F7F7Fu : f8_pack4(o[0], o[1], o[2], o[3], inv),
                     bad ? 0x7F7F7F7Fu : f8_pack4(o[4], o[5], o[6], o[7], inv)};
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + row * 128 + 8 * i) = w;
    if (i == 0) {
      const int SC = (int)f8_scale_cols((int64_t)a.Hq * 128);
      uint8_t* const at = a.scales + (int64_t)b * SC;
      at[head] = (uint8_t)byte;
      if (head == a.Hq - 1)
        for (int c = a.Hq; c < SC; ++c) at[c] = 0;
    }
  } else if (8 * i < D) {
    *reinterpret_cast<v4u*>(static_cast<uint8_t*>(a.out) + (row * D + 8 * i) * 2) =
        v4u{pack2_16<BF16>(o[0], o[1]), pack2_16<BF16>(o[2], o[3]), pack2_16<BF16>(o[4], o[5]), pack2_16<BF16>(o[6], o[7])};
  }
}

// A row's sixteen lanes' eight values each: a cached row's values d = 8 i .. + 7 in float32 (not scaled).
template <bool BF16, bool WIDE>
__device__ __forceinline__ void cached_8(const uint8_t* row, int i, float* x) {
  if constexpr (WIDE) {
    unpack8_16<BF16>(*reinterpret_cast<const v4u*>(row + 16 * i), x);
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(row + 8 * i);
    unpack8_16<true>(widen8<true>(w.x, w.y), x);
  }
}

// One head's sum over the keys [begin, end) of sequence b again, by the definition, one weight and one product a key.  For
// sums that are not finite: with a weight as a sum of 16-bit numbers, of which all but the first may be negative or zero,
// a value that is infinite comes out as NaN.  Sixteen lanes a head, values d = 8 i .. + 7 in sum; the maximum in m, the sum of
// weights (2^lift larger, as the pieces' are) in l.  Slow, some 70 instructions a key (one infinite value takes a call of 513
// tokens, 32 / 8 heads of 128, from 12 to 276 us, of 37 sequences of 50 to 4000 from 54 to 847), and small.
template <bool BF16, bool WIDE>
__device__ __forceinline__ void keys_again(const PagedArgs& a, int b, int head, int begin, int end, float lift, int i, float& m,
                                           float& l, float* sum) {
  const Pages& c = a.c;
  const int RB = WIDE ? 2 * c.D : c.D, hk = head / (a.Hq / c.Hkv);
  const bool there = 8 * i < c.D;
  float q[8], x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) q[e] = x[e] = sum[e] = 0.0f;
  if (there) unpack8_16<BF16>(*reinterpret_cast<const v4u*>(a.q + b * a.qs + head * a.qh + 16 * i), q);
  m = -INFINITY, l = 0.0f;
#pragma unroll 1
  for (int key = begin; key < end; ++key) {
    const int page = c.table[(int64_t)b * c.width + key / c.page];
    if (page < 0 || page >= c.pages) continue;
    const int64_t row = ((int64_t)page * c.Hkv + hk) * c.page + key % c.page;
    if (there) cached_8<BF16, WIDE>(c.k + row * RB, i, x);
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(x[e], q[e], s);
    s = row16_sum(s);
    if constexpr (!WIDE) s *= e8m0_value(c.ks[row]);
    s *= a.scale;
    const float to = fmaxf(m, s), base = to == -INFINITY ? 0.0f : to;
    const float f = __builtin_amdgcn_exp2f(m - base);
    float w = __builtin_amdgcn_exp2f(s - base + lift);
    m = to;
    l = fmaf(l, f, w);
    if constexpr (!WIDE) w *= e8m0_value(c.vs[row]);
    if (there) cached_8<BF16, WIDE>(c.v + row * RB, i, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = fmaf(w, x[e], sum[e] * f);
  }
}

// Floats of a partial result: 16 heads' sums, then their maxima and their sums of weights.
template <int DP> constexpr int PART = 16 * DP + 32;

// Wavefronts of a workgroup and workgroups on a compute unit, which together fill its LDS with rings.  (Four wavefronts and
// half as many workgroups wait longer at a piece's end: 37 sequences of 50 to 4000 in 16 bits 70 and 64 us, 160 of 200 to
// 8000 in 8 bits 261 and 250; one wavefront each leaves more to join, two of 131072 in 8 bits 112 and 107.)
constexpr int NW = 2;
constexpr int resident(bool wide, int DP) { return wide && DP == 128 ? 2 : wide || DP == 128 ? 4 : 8; }

// A row of rows that has no page.
constexpr uint32_t NOWHERE = 0xFFFFFFFFu;

// BF16: of queries and outputs.  WIDE: 16-bit rows of that type, else E4M3.  DP: D rounded up.  RES: workgroups
// on a compute unit.
// WHOLE: a run is a unit, without looking at the other sequences' lengths; nothing is left to be joined.
template <bool BF16, bool WIDE, int DP, int NW, int RES, bool WHOLE>
__global__ __launch_bounds__(64 * NW, RES) void paged_kernel(PagedArgs a, int W) {
  constexpr int BLK = 32 * NW;                               // keys of a block
  constexpr int PITCH = WIDE ? 2 * DP : DP;                  // bytes of a row in LDS
  constexpr int CH = PITCH / 16;                             // its 16-byte chunks
  constexpr int LOADS = 16 * PITCH / 1024;                   // of 16 rows
  constexpr int SLOT = 64 * PITCH + (WIDE ? 0 : 128);        // 32 keys, 32 values, scales
  constexpr int NV = 4 * LOADS + (WIDE ? 0 : 1);             // vector loads of a block
  constexpr int KS = DP / 32, DT = DP / 16;
  constexpr int RING = 2 * SLOT;
  constexpr bool PB = BF16 || !WIDE;                         // the weights' 16-bit type
  constexpr int NUMBERS = PB ? 3 : 2;                          // of a weight
  constexpr float LIFT = PB ? 0.0f : 6.0f;
  static_assert(PART<DP> * 4 <= SLOT, "a slot takes a wavefront's results");
  __shared__ __align__(1024) uint8_t lds[NW * RING];
  const Pages& c = a.c;
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int G = a.Hq / c.Hkv, HC = (G + 15) / 16, HH = c.Hkv * HC;
  const int RB = WIDE ? 2 * c.D : c.D;                       // bytes of a row
  const int w = blockIdx.x;
  Run* const runs = reinterpret_cast<Run*>(a.part + (int64_t)2 * W * PART<DP>);

  Piece p;
  int64_t left;
  if (WHOLE) {
    p.b = w / HH, p.unit = w % HH, p.j0 = 0;
    p.len = length_of(c, p.b);
    left = p.j1 = p.nb = blocks_in<NW>(p.len);
    if (left == 0) {                                         // no keys: zeros
      const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int i = 16 * (p.unit % HC) + (threadIdx.x >> 4); i < min(G, 16 * (p.unit % HC + 1)); i += 4 * NW)
        store_row<BF16>(zero, a, p.b, p.unit / HC * G + i, threadIdx.x & 15);
      return;
    }
  } else {
    int64_t N;
    left = find_run<NW>(c, HH, w, W, N, p);
    if (threadIdx.x == 0) runs[w] = left > 0 ? Run{N, p.b, p.unit, p.j0, p.nb, {0, 0}} : Run{N, 0, 0, 0, 0, {0, 0}};
    if (left == 0) return;
  }

  auto swizzle_k = [](int row) { return PITCH == 256 ? row & 15 : PITCH == 128 ? (row >> 1) & 7 : (row >> 2) & 3; };
  auto swizzle_v = [](int row) {
    if (!WIDE) return PITCH == 128 ? (row >> 1) & 7 : (row >> 2) & 3;
    return PITCH == 256 ? 2 * (row & 7) : PITCH == 128 ? 2 * ((row >> 1) & 3) : 2 * ((row >> 2) & 1);
  };
  // this lane's part of a 1024-byte load: offsets of its key and value chunks from the row of the load
  int vk[LOADS], vv[LOADS];
#pragma unroll
  for (int n = 0; n < LOADS; ++n) {
    const int row = n * (1024 / PITCH) + lane / CH, ch = lane % CH;
    const int ck = ch ^ swizzle_k(row), cv = ch ^ swizzle_v(row);
    vk[n] = 16 * ck < RB ? row * RB + 16 * ck : KQ_OOB;
    vv[n] = 16 * cv < RB ? row * RB + 16 * cv : KQ_OOB;
  }
  const uint32_t ring0 = lds_addr(lds) + wid * RING;
  const uint8_t* const ring = lds + wid * RING;

  // Where the cache has the wavefront's keys of 32 blocks from j on: lane i has the sixteenth of the row of key
  // 16 (i % 2) of block j + i / 2 (pages are multiples of 16 rows).
  auto rows_of = [&](const Piece& p, int j) {
    const int64_t key = (int64_t)BLK * (j + (lane >> 1)) + 32 * wid + 16 * (lane & 1);
    uint32_t at = NOWHERE;
    if (key < p.len && j + (lane >> 1) < p.j1) {
      const int k = (int)key, page = c.table[(int64_t)p.b * c.width + k / c.page];
      if (page >= 0 && page < c.pages)
        at = (uint32_t)((((int64_t)page * c.Hkv + p.unit / HC) * c.page + k % c.page) >> 4);
    }
    return at;
  };
  // the wavefront's 32 keys of block j; n: how many of each 16 there are
  auto load = [&](int slot, const Piece& p, int j, uint32_t rows, int first, int (&n)[2]) {
    const uint32_t at = ring0 + slot * SLOT;
    int64_t row[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t r16 = __builtin_amdgcn_readlane(rows, 2 * (j - first) + s);
      n[s] = r16 == NOWHERE ? 0 : min(16, p.len - (BLK * j + 32 * wid + 16 * s));
      row[s] = r16 == NOWHERE ? 0 : (int64_t)r16 * 16;
      const v4i rk = rsrc_words(c.k + row[s] * RB, (int64_t)n[s] * RB), rv = rsrc_words(c.v + row[s] * RB, (int64_t)n[s] * RB);
#pragma unroll
      for (int i = 0; i < LOADS; ++i) lds_load16(rk, at + 16 * PITCH * s + 1024 * i, vk[i]);
#pragma unroll
      for (int i = 0; i < LOADS; ++i) lds_load16(rv, at + 16 * PITCH * (2 + s) + 1024 * i, vv[i]);
    }
    if constexpr (!WIDE) {
      if (lane < 4) lds_load16_at(at + 64 * PITCH, (lane < 2 ? c.ks : c.vs) + ((lane & 1) ? row[1] : row[0]));
    }
  };
  // queries: this lane's column is head r of the unit; 8-bit rows give a lane 16 codes at a time, which are two
  // products' worth
  auto queries = [&](const Piece& p, v4u (&q)[KS]) {
    const int h0 = 16 * (p.unit % HC);
    const uint8_t* const at = a.q + p.b * a.qs + (int64_t)(p.unit / HC * G + h0 + r) * a.qh;
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      const int d = WIDE ? 32 * i + 8 * g : 64 * (i / 2) + 16 * g + 8 * (i % 2);
      q[i] = v4u{0, 0, 0, 0};
      if (h0 + r < G && d < c.D) q[i] = *reinterpret_cast<const v4u*>(at + 2 * d);
    }
  };

  uint32_t rows = rows_of(p, p.j0), rows2 = 0;
  int first = p.j0;
  v4u q[KS], q2[KS];
  queries(p, q);
  int n[2], n2[2], slot = 0;
  load(0, p, p.j0, rows, first, n);
  bool first_piece = true;
  for (;;) {
    // the piece after this one, and what its first block needs
    Piece p2 = p;
    left -= p.j1 - p.j0;
    if (left > 0) {
      p2.j0 = 0;
      if (++p2.unit == HH) {
        p2.unit = 0;
        do {
          if (++p2.b >= c.B) return;
          p2.len = length_of(c, p2.b);
          p2.nb = blocks_in<NW>(p2.len);
        } while (p2.nb == 0);
      }
      p2.j1 = (int)min((int64_t)p2.nb, left);
      rows2 = rows_of(p2, 0);
      queries(p2, q2);
    }
    v4f acc[DT];
#pragma unroll
    for (int i = 0; i < DT; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.0f;
    for (int j = p.j0; j < p.j1; ++j) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");     // the slot that is filled next has been read
      if (j + 1 < p.j1) {
        if (j + 1 == first + 32) first = j + 1, rows = rows_of(p, first);
        load(slot ^ 1, p, j + 1, rows, first, n2);
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(NV));
      } else if (left > 0) {
        load(slot ^ 1, p2, 0, rows2, 0, n2);
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(NV));
      } else {
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
      }
      asm volatile("" ::: "memory");
      const uint8_t* const sk = ring + slot * SLOT;
      const uint8_t* const sv = sk + 32 * PITCH;
      v4f t[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) t[s] = v4f{0.f, 0.f, 0.f, 0.f};
      if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
          for (int s = 0; s < 2; ++s)
            t[s] = mfma16<BF16>(
                *reinterpret_cast<const v4u*>(sk + PITCH * (16 * s + r) + 16 * ((4 * i + g) ^ swizzle_k(r))), q[i], t[s]);
      } else {
#pragma unroll
        for (int i = 0; i < KS / 2; ++i)
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const v4u k16 = *reinterpret_cast<const v4u*>(sk + PITCH * (16 * s + r) + 16 * ((4 * i + g) ^ swizzle_k(r)));
            t[s] = mfma16<BF16>(widen8<BF16>(k16[0], k16[1]), q[2 * i], t[s]);
            t[s] = mfma16<BF16>(widen8<BF16>(k16[2], k16[3]), q[2 * i + 1], t[s]);
          }
      }
      float scale[16];                                       // of the lane's eight keys, then of its values
      float* const vscale = scale + 8;
      if constexpr (!WIDE) {
        const uint32_t* const bytes = reinterpret_cast<const uint32_t*>(sk + 64 * PITCH + 4 * g);
        e8m0_values({bytes[0], bytes[4], bytes[8], bytes[12]}, scale);
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e / 4][e & 3] *= scale[e];
      }
      if (n[0] + n[1] < 32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool seen = 4 * g + (e & 3) < (e < 4 ? n[0] : n[1]);
          t[e / 4][e & 3] = seen ? t[e / 4][e & 3] : -INFINITY;
          if constexpr (!WIDE) vscale[e] = seen ? vscale[e] : 0.0f;
        }
      }
      float top = -INFINITY;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, t[e / 4][e & 3]);
      top = half_max(row_pair_max(top)) * a.scale;
      if (__any(top > m + 8.0f)) {
        const float to = fmaxf(m, top);
        const float f = to == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - to);
        m = to;
        l *= f;
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][e] *= f;
      }
      const float base = (m == -INFINITY ? 0.0f : m) - LIFT;
      float pr[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        pr[e] = __builtin_amdgcn_exp2f(fmaf(t[e / 4][e & 3], a.scale, -base));
        l += pr[e];
        if constexpr (!WIDE) pr[e] *= vscale[e];
      }
      // a weight is a sum of 16-bit numbers: relative error 2^-24 (three of bf16), 2^-22 (two of fp16; or 2^-31 of the
      // largest, as they are held 2^LIFT larger, to 2^14 at most)
      v4u wn[NUMBERS];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int u = 0; u < NUMBERS; ++u) {
          const uint32_t w = pack2_16<PB>(pr[2 * e], pr[2 * e + 1]);
          wn[u][e] = w;
          pr[2 * e] -= unpack1_16<PB>((uint16_t)w), pr[2 * e + 1] -= unpack1_16<PB>((uint16_t)(w >> 16));
        }
      }
#pragma unroll
      for (int i = 0; i < DT; ++i) {
        v4u v;
        if constexpr (WIDE) {
          const int row = 4 * g + (r >> 2);
          const uint8_t* const at = sv + PITCH * row + 16 * ((2 * i + ((r & 3) >> 1)) ^ swizzle_v(row)) + 8 * (r & 1);
          const v2u v0 = lds_tr16(at), v1 = lds_tr16(at + 16 * PITCH);
          v = v4u{v0[0], v0[1], v1[0], v1[1]};
        } else {
          const int k = r >> 1, row = 4 * g + (k & 3) + 16 * (k >> 2);
          const v2u w8 = lds_tr8(sv + PITCH * row + 16 * (i ^ swizzle_v(row)) + 8 * (r & 1));
          v = widen8<true>(w8[0], w8[1]);
        }
#pragma unroll
        for (int u = 0; u < NUMBERS; ++u) acc[i] = mfma16<PB>(v, wn[u], acc[i]);
      }
      slot ^= 1;
      n[0] = n2[0], n[1] = n2[1];
    }
    // the wavefronts' results meet in the slots that were read last; the others are being filled
    const int done = slot ^ 1;
    l = half_sum(row_pair_sum(l));
    {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      float* const o = reinterpret_cast<float*>(lds + wid * RING + done * SLOT);
#pragma unroll
      for (int i = 0; i < DT; ++i) *reinterpret_cast<v4f*>(o + DP * r + 16 * i + 4 * g) = acc[i];
      if (g == 0) o[16 * DP + r] = m, o[16 * DP + 16 + r] = l;
    }
    lds_barrier();
    // thread: head threadIdx / 16, values 8 i .. + 7
    for (int hd = threadIdx.x >> 4; hd < min(16, G - 16 * (p.unit % HC)); hd += 4 * NW) {
      const int i = threadIdx.x & 15;
      const float* o[NW];
      float top = -INFINITY, total = 0.0f, sum[8];
#pragma unroll
      for (int u = 0; u < NW; ++u) {
        o[u] = reinterpret_cast<const float*>(lds + u * RING + done * SLOT);
        top = fmaxf(top, o[u][16 * DP + hd]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
#pragma unroll
      for (int u = 0; u < NW; ++u) {
        const float mu = o[u][16 * DP + hd];
        const float f = mu == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mu - top);
        total = fmaf(f, o[u][16 * DP + 16 + hd], total);
        if (8 * i < DP) {
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[e] = fmaf(f, o[u][DP * hd + 8 * i + e], sum[e]);
        }
      }
      const int head = p.unit / HC * G + 16 * (p.unit % HC) + hd;
      float zero = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) zero = fmaf(sum[e], 0.0f, zero);
      if (__builtin_expect(__any(!(zero == 0.0f)), 0))
        keys_again<BF16, WIDE>(a, p.b, head, BLK * p.j0, (int)min((int64_t)p.len, (int64_t)BLK * p.j1), LIFT, i, top, total, sum);
      if (WHOLE || (p.j0 == 0 && p.j1 == p.nb)) {
        const float inv = 1.0f / total;                      // no weight: zeros, whatever the values
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = total == 0.0f ? 0.0f : sum[e] * inv;
        store_row<BF16>(sum, a, p.b, head, i);
      } else {
        float* const part = a.part + (int64_t)(2 * w + (first_piece ? 0 : 1)) * PART<DP>;
        if (8 * i < DP) {
#pragma unroll
          for (int e = 0; e < 8; e += 4)
            *reinterpret_cast<v4f*>(part + DP * hd + 8 * i + e) = v4f{sum[e], sum[e + 1], sum[e + 2], sum[e + 3]};
        }
        if (i == 0) part[16 * DP + hd] = top, part[16 * DP + 16 + hd] = total;
      }
    }
    if (left == 0) return;
    lds_barrier();                                           // before the slots are filled again
    first_piece = false;
    p = p2;
    rows = rows2;
    first = 0;
#pragma unroll
    for (int i = 0; i < KS; ++i) q[i] = q2[i];
  }
}

// Joins what the runs left of units they share; ROWS rows of 16 threads take a unit's runs in turn for each head, four at a
// time.  ROWS = 4 (many units): each run that begins inside a unit (the first of those in it) is a workgroup's,
// for four of the unit's heads, and further workgroups write zeros for the sequences without keys, 64 each.
// ROWS = 16 (many runs of each unit): a workgroup for each unit and head.
template <bool BF16, int DP, int ROWS>
__global__ __launch_bounds__(256) void paged_join_kernel(PagedArgs a, int W, int groups) {
  constexpr int HEADS = 16 / ROWS, AT = 4;
  __shared__ float so[16][DP + 2];
  const Pages& c = a.c;
  const int G = a.Hq / c.Hkv, HC = (G + 15) / 16, HH = c.Hkv * HC;
  const int k = threadIdx.x >> 4, i = threadIdx.x & 15, lane = threadIdx.x & 63;
  float sum[8], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
  const int hd = blockIdx.x % groups * HEADS + k / ROWS;
  int64_t N, x0, begin;                                      // all blocks; the unit's first; its first run's first
  int b, unit, nb, w0;                                       // w0: the unit's first run
  if constexpr (ROWS == 4) {
    if (blockIdx.x >= (uint32_t)((W - 1) * groups)) {
      const int b0 = 64 * (blockIdx.x - (W - 1) * groups);
      uint64_t none = __ballot(b0 + lane < c.B && c.lengths[b0 + lane] <= 0);
      for (; none; none &= none - 1)
        for (int h = k; h < a.Hq; h += 16) store_row<BF16>(sum, a, b0 + __builtin_ctzll(none), h, i);
      return;
    }
    const int w = blockIdx.x / groups + 1;
    const Run* const runs = reinterpret_cast<const Run*>(a.part + (int64_t)2 * W * PART<DP>);
    N = runs[0].N;
    const Run u = runs[w];
    W = (int)min((int64_t)W, N);
    if (w >= W || u.j0 == 0) return;
    x0 = run_start(w, N, W) - u.j0;
    w0 = w - 1;
    begin = run_start(w0, N, W);
    if (begin > x0) return;                                  // the run before began inside it, too
    b = u.b, unit = u.unit, nb = u.nb;
  } else {
    const int at = blockIdx.x / groups;
    b = at / HH, unit = at % HH;
    uint32_t before = 0, all = 0, own = 0;
    for (int b0 = 0; b0 < c.B; b0 += 64) {
      const uint32_t n = b0 + lane < c.B ? blocks_in<NW>(held(c, c.lengths[b0 + lane])) : 0;
      all += n;
      before += b0 + lane < b ? n : 0;
      own += b0 + lane == b ? n : 0;
    }
    N = (int64_t)(uint32_t)__builtin_amdgcn_readlane(wave_scan(all), 63) * HH;
    nb = __builtin_amdgcn_readlane(wave_scan(own), 63);
    if (nb == 0) {                                           // no keys: zeros
      if (k == 0 && hd < min(16, G - 16 * (unit % HC))) store_row<BF16>(sum, a, b, unit / HC * G + 16 * (unit % HC) + hd, i);
      return;
    }
    W = (int)min((int64_t)W, N);
    x0 = (int64_t)(uint32_t)__builtin_amdgcn_readlane(wave_scan(before), 63) * HH + (int64_t)unit * nb;
    w0 = (int)(((x0 + 1) * W - 1) / N);
    begin = run_start(w0, N, W);
    if (run_start(w0 + 1, N, W) >= x0 + nb) return;          // one run has it all
  }
  const int h0 = 16 * (unit % HC);
  // the last run with a block of the unit: ((x + 1) W - 1) / N for its last block x
  const int last = (int)(((x0 + nb) * W - 1) / N);
  if (hd < min(16, G - h0)) {
    for (int v0 = w0 + k % ROWS; v0 <= last; v0 += ROWS * AT) {
      float mv[AT], lv[AT];
      v4f ov[AT][2];
#pragma unroll
      for (int t = 0; t < AT; ++t) {
        const int v = v0 + ROWS * t;
        mv[t] = -INFINITY, lv[t] = 0.0f;
        ov[t][0] = ov[t][1] = v4f{0.f, 0.f, 0.f, 0.f};
        if (v <= last) {
          const float* const part = a.part + (int64_t)(2 * v + (v == w0 && begin < x0 ? 1 : 0)) * PART<DP>;
          mv[t] = part[16 * DP + hd], lv[t] = part[16 * DP + 16 + hd];
          if (8 * i < DP) {
            ov[t][0] = *reinterpret_cast<const v4f*>(part + DP * hd + 8 * i);
            ov[t][1] = *reinterpret_cast<const v4f*>(part + DP * hd + 8 * i + 4);
          }
        }
      }
      float to = m;
#pragma unroll
      for (int t = 0; t < AT; ++t) to = fmaxf(to, mv[t]);
      const float f = to == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - to);
      m = to;
      l *= f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] *= f;
#pragma unroll
      for (int t = 0; t < AT; ++t) {
        const float ft = mv[t] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mv[t] - to);
        l = fmaf(ft, lv[t], l);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = fmaf(ft, ov[t][e / 4][e % 4], sum[e]);
      }
    }
  }
  if (8 * i < DP) {
#pragma unroll
    for (int e = 0; e < 8; ++e) so[k][8 * i + e] = sum[e];
  }
  if (i == 0) so[k][DP] = m, so[k][DP + 1] = l;
  __syncthreads();
  if (k % ROWS > 0 || hd >= min(16, G - h0)) return;
  float top = -INFINITY, total = 0.0f;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) top = fmaxf(top, so[k + r][DP]);
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const float f = so[k + r][DP] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(so[k + r][DP] - top);
    total = fmaf(f, so[k + r][DP + 1], total);
    if (8 * i < DP) {
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] = fmaf(f, so[k + r][8 * i + e], sum[e]);
    }
  }
  const float inv = 1.0f / total;                            // no weight: zeros, whatever the values
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = total == 0.0f ? 0.0f : sum[e] * inv;
  store_row<BF16>(sum, a, b, unit / HC * G + h0 + hd, i);
}

template <bool BF16, int DP, int ROWS>
hipError_t join(const PagedArgs& a, int W, int64_t units, int heads, hipStream_t s) {
  const int groups = (heads + 16 / ROWS - 1) / (16 / ROWS);
  const int64_t grid = ROWS == 4 ? (int64_t)(W - 1) * groups + (a.c.B + 63) / 64 : units * groups;
  hipLaunchKernelGGL((paged_join_kernel<BF16, DP, ROWS>), dim3((unsigned)grid), dim3(256), 0, s, a, W, groups);
  return hipGetLastError();
}

// HBM bounds long fillings (8192 tokens of 8 heads of 128 to 8 bits, 50 MB: 12 us), a launch and two loads in turn the small
// ones (37 tokens 3.7 us).  One wavefront a token: its sequence, position and page, then the rows of its heads, four at a time, 16
// lanes a row; 8-bit rows are quantized as a group (row16_umax, as the quantizer's).
template <bool BF16, bool WIDE>
__global__ __launch_bounds__(256) void cache_append_kernel(AppendArgs a) {
  const int lane = threadIdx.x & 63;
  const Pages& c = a.c;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= a.T) return;
  int64_t b = t, behind = 1;                                 // tokens of the sequence from this one on
  if (a.cu) {
    b = last_before(c.B, [&](int i) { return a.cu[i] <= t; });
    if (t < a.cu[b] || t >= a.cu[b + 1]) return;
    behind = a.cu[b + 1] - t;
  }
  const int64_t at = (int64_t)c.lengths[b] - behind;
  if (at < 0 || at >= (int64_t)c.width * c.page) return;
  const int64_t page = c.table[b * c.width + at / c.page];
  if (page < 0 || page >= c.pages) return;
  const int sub = lane & 15, RB = WIDE ? 2 * c.D : c.D;
  for (int r0 = 0; r0 < 2 * c.Hkv; r0 += 4) {
    const int row = r0 + (lane >> 4);
    const bool key = row < c.Hkv;
    const int h = key ? row : row - c.Hkv;
    const bool there = row < 2 * c.Hkv && 8 * sub < c.D;
    v4u w = {0, 0, 0, 0};
    if (there) {
      const AttnRows& src = key ? a.k : a.v;
      w = *reinterpret_cast<const v4u*>(src.p + t * src.ts + h * src.hs + 16 * sub);
    }
    const int64_t to = (page * c.Hkv + h) * c.page + at % c.page;
    if constexpr (WIDE) {
      if (there) *reinterpret_cast<v4u*>((key ? c.k : c.v) + to * RB + 16 * sub) = w;
    } else {
      float y[8];
      unpack8_16<BF16>(w, y);
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = umax32(top, abs_bits(y[e]));
      const uint32_t byte = f8_scale_byte(row16_umax(top));
      const bool bad = byte == 255u;
      const float inv = bad ? 1.0f : f8_inv_scale(byte);
      if (there) {
        *reinterpret_cast<uint2*>((key ? c.k : c.v) + to * RB + 8 * sub) =
            uint2{bad ? 0x7F7F7F7Fu : f8_pack4(y[0], y[1], y[2], y[3], inv),
                  bad ? 0x7F7F7F7Fu : f8_pack4(y[4], y[5], y[6], y[7], inv)};
        if (sub == 0) (key ? c.ks : c.vs)[to] = (uint8_t)byte;
      }
    }
  }
}

// A unit is one workgroup's, and nothing is joined (so no workspace is needed), where tables hold up to 640 keys, or up to 2048 and there is a unit
// for every compute unit: 32 / 8 heads of 128, whole and dealt (us): one sequence of 500 9.4 and 9.6, 1000 14 and 9.9; 8 of
// 1000 16.3 and 15.7; 64 of 0 to 2000 in 8 bits 38 and 44; 300 of 100 in 16 bits 43 and 46; 160 of 200 to 8000 in 8 bits 281 and
// 250.  Four wavefronts then, so that a unit is sooner done, or two where the units fill the chip (300 of 0 to 1000: 130
// and 148; 64 of 500 in 8 bits the other way, 21 and 19).
bool whole(int64_t units, int64_t longest) { return longest <= 640 || (longest <= 2048 && units >= device_cu_count()); }

// Runs of a call: one for each workgroup that the compute units hold, and no more than blocks.
int64_t runs(int64_t B, int Hq, int Hkv, int64_t longest, bool wide, int DP) {
  const int G = Hq / Hkv, HC = (G + 15) / 16, block = 32 * NW;
  const int64_t blocks = B * Hkv * HC * ((longest + block - 1) / block);
  const int64_t most = (int64_t)device_cu_count() * resident(wide, DP);
  return blocks < 1 ? 1 : blocks < most ? blocks : most;
}

template <bool BF16, bool WIDE, int DP>
hipError_t go(const PagedArgs& a, hipStream_t s) {
  constexpr int RES = resident(WIDE, DP);
  const int64_t longest = (int64_t)a.c.width * a.c.page;
  const int G = a.Hq / a.c.Hkv, HC = (G + 15) / 16;
  const int64_t units = (int64_t)a.c.B * a.c.Hkv * HC;
  if (whole(units, longest)) {
    if (units >= (int64_t)device_cu_count() * RES)
      hipLaunchKernelGGL((paged_kernel<BF16, WIDE, DP, 2, RES, true>), dim3((unsigned)units), dim3(128), 0, s, a, 0);
    else
      hipLaunchKernelGGL((paged_kernel<BF16, WIDE, DP, 4, RES / 2, true>), dim3((unsigned)units), dim3(256), 0, s, a, 0);
    return hipGetLastError();
  }
  const int W = (int)runs(a.c.B, a.Hq, a.c.Hkv, longest, WIDE, DP);
  hipLaunchKernelGGL((paged_kernel<BF16, WIDE, DP, NW, RES, false>), dim3(W), dim3(64 * NW), 0, s, a, W);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int heads = G < 16 ? G : 16;
  // many runs of each unit: 16 at once for a head; else as few workgroups as there can be (1023 joins 10 and 5 us)
  return W > 16 * units ? join<BF16, DP, 16>(a, W, units, heads, s) : join<BF16, DP, 4>(a, W, units, heads, s);
}

}  // namespace

// For both kinds of cache.
size_t paged_workspace_bytes(int64_t B, int Hq, int Hkv, int D, int64_t longest) {
  if (whole(B * Hkv * ((Hq / Hkv + 15) / 16), longest)) return 0;
  const int DP = D <= 64 ? 64 : 128;
  const int64_t part = DP == 64 ? PART<64> : PART<128>;
  const int64_t a = runs(B, Hq, Hkv, longest, false, DP), b = runs(B, Hq, Hkv, longest, true, DP);
  return (size_t)(a > b ? a : b) * (2 * part * sizeof(float) + sizeof(Run));
}

hipError_t launch_paged_attention(bool bf16, bool wide, const PagedArgs& a, hipStream_t s) {
  if (a.c.D <= 64) {
    if (bf16) return wide ? go<true, true, 64>(a, s) : go<true, false, 64>(a, s);
    return wide ? go<false, true, 64>(a, s) : go<false, false, 64>(a, s);
  }
  if (bf16) return wide ? go<true, true, 128>(a, s) : go<true, false, 128>(a, s);
  return wide ? go<false, true, 128>(a, s) : go<false, false, 128>(a, s);
}

hipError_t launch_cache_append(bool bf16, bool wide, const AppendArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.T + 3) / 4)), block(256);
  if (bf16 && wide) hipLaunchKernelGGL((cache_append_kernel<true, true>), grid, block, 0, s, a);
  else if (bf16) hipLaunchKernelGGL((cache_append_kernel<true, false>), grid, block, 0, s, a);
  else if (wide) hipLaunchKernelGGL((cache_append_kernel<false, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((cache_append_kernel<false, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace kq
