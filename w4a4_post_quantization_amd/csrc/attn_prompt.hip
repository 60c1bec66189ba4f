// Attention of packed sequences: o_i = sum_j p_ij v_j, p the softmax over the visible keys j of
// scale q_i . k_j (causal: j <= i + Lk - Lq), in one pass with the running maximum and sum.
//
// A workgroup takes 32 NW queries of one head, 32 to a wavefront, and walks the keys in tiles of 64
// that are loaded straight into LDS, the next tile under the present one's products.  Everything is
// kept transposed, a query a column: S^T = K Q^T leaves a lane with 32 of the 64 scores of ONE query
// (the other 32 are in the lane 32 away), so the maximum takes one exchange, the sum none until the
// end, and the weights are already the second product's operand: O^T += V^T P^T contracts over keys
// in whatever order both operands share, here the order in which the scores came out, and V^T comes
// from LDS by transposing reads.
//
// The running maximum is only moved when a score passes it by 2^8 (weights up to 256 lose nothing in
// float32 sums or 16-bit weights), which spares most rescalings of the 16 DT accumulators.  fp16 weights are held
// 2^6 larger, to 2^14 at most, so that what falls under fp16's smallest step is 2^-31 of the largest.
//
// The weights are rounded to the 16-bit type for the second product, which keeps it one matrix instruction; 16-bit outputs
// show little of it (relative error against 64 bits 1.76e-3 bf16, 2.20e-4 fp16; of float32 throughout 1.66e-3 and
// 2.08e-4), codes fall to the other side of a rounding border here and there (0.6 to 1% of the norm bf16, 0.2% fp16; E4M3
// itself 2.7%).  PRECISE multiplies a weight as a sum of 16-bit numbers, two of fp16 or three of bf16, as exactly as float32
// holds it: 1.66e-3 and 2.08e-4, codes 0.015 to 0.026% (float32 throughout: 0.017 and 0.023).  8192 tokens of 32 / 8 heads of
// 128 in bf16 take 938 us so and not 510 (with two numbers 693, codes 0.027%, which is measurably more than float32's), two
// images of 4096 with 16 heads of 72 in fp16 300 and not 210, 37 tokens 9.6 and not 8.6.
//
// A step multiplies the next tile's keys while the present tile's exponentials are taken, and the present
// tile's values while the next maximum is, so that the matrix cores and the vector units have work of
// the same wavefront side by side.
// Long prompts are bound by the chip's power: 8192 tokens, 32 / 8 heads of 128, causal, bf16 take 495 to 546 us (1.01 to
// 1.11 PFLOP/s; a library product of 8192^3 1.41) with the matrix cores 63% busy at 1.54 GHz, so what is left
// out counts more than what is hidden: of that time exponentials have 5%, the fragments' LDS reads 11%, the tiles' loads
// 6 to 8%, barriers 1%.  Short ones are bound by latency: 37 tokens 8.4 us, of which a launch and three loads in turn.
#include "kq_attn.hpp"
#include "kq_launch.hpp"

#include <type_traits>

namespace kq {

namespace {

constexpr int KT = 64;                 // keys of a tile

// Where a workgroup's queries and keys are.  Its rows are those of one key head: row i is query i / G of head
// i % G of the G that share the key head, so that they share the tiles of keys, too, and a tile's rows
// end at nearly the same key.
struct Span {
  int64_t q0, k0;                      // first query of the sequence, first key
  int32_t nq, nk;                      // their numbers
  int32_t first;                       // the workgroup's first row within the sequence
};

// Sequence i's rows begin at slot G cu_q[i] / QT + i of the grid, which leaves each at least as many
// slots as it has tiles without anyone having summed the tiles: a slot finds its sequence by the
// starts up to itself, looking at 64 at a time (4000 sequences of 9 tokens, 8 / 2 heads of 64: 61 us;
// looking at all of them took 151).  Entries are held to 0 .. T and to their order.
template <int QT>
__device__ bool find_span(const AttnArgs& a, int G, int32_t slot, Span& s) {
  if (!a.cu_q) {
    s = {0, 0, (int32_t)a.T, (int32_t)a.Tk, slot * QT};
    return true;
  }
  const int lane = threadIdx.x & 63;
  const int32_t T = (int32_t)a.T, Tk = (int32_t)a.Tk;
  auto start = [&](int32_t q, int i) { return min(max(q, 0), T) * G / QT + i; };
  int lo = 0, len = a.B;
  narrow(lo, len, [&](int i) { return start(a.cu_q[i], i) <= slot; });
  // lane l: candidate lo + l's four entries, so that up to 64 sequences take one load
  const int at = lo + min(lane, len - 1);
  const int32_t lq0 = a.cu_q[at], lq1 = a.cu_q[at + 1], lk0 = a.cu_k[at], lk1 = a.cu_k[at + 1];
  const int found = __popcll(__ballot(lane < len && start(lq0, at) <= slot));  // as an int: it may be 0, less 1
  const int l = found > 0 ? found - 1 : 0, i = lo + l;
  int32_t q0 = __builtin_amdgcn_readlane(lq0, l), q1 = __builtin_amdgcn_readlane(lq1, l);
  int32_t k0 = __builtin_amdgcn_readlane(lk0, l), k1 = __builtin_amdgcn_readlane(lk1, l);
  q0 = min(max(q0, 0), T), q1 = min(max(q1, q0), T);
  k0 = min(max(k0, 0), Tk), k1 = min(max(k1, k0), Tk);
  const int tile = slot - (q0 * G / QT + i);                 // below 0 for no sequence, and by entries out of order
  s = {q0, k0, q1 - q0, k1 - k0, tile * QT};
  return tile >= 0 && s.first < s.nq * G;
}

// acc + both halves of a packed pair (their products by 1 are exact).
template <bool BF16>
__device__ __forceinline__ float add_pair(uint32_t w, float acc) {
  if constexpr (BF16) {
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(v2bf, w), __builtin_bit_cast(v2bf, 0x3F803F80u), acc, false);
  } else {
    return add_f16x2(w, acc);
  }
}

// Scores of masked keys.
constexpr float HIDDEN = -INFINITY;

// PRECISE: a weight is multiplied as the sum of several 16-bit numbers, else rounded to one.
template <bool BF16, int KS, int DT, int NW, bool PRECISE>
struct Prompt {
  static constexpr int QT = 32 * NW;
  static constexpr float LIFT = BF16 ? 0.0f : 6.0f;
  static constexpr int NUMBERS = BF16 ? 3 : 2;                         // of a precise weight: 24 or 22 bits
  static constexpr int PITCH = KS <= 4 ? 128 : 256;                  // bytes of a key's row in LDS
  static constexpr int TILE = KT * PITCH;
  static constexpr int LOADS = TILE / (1024 * NW);                   // of a wavefront, a matrix and tile
  static constexpr int ROWS = 1024 / PITCH;                          // rows of a load
  static constexpr int OPITCH = 64 * DT + 16;                        // bytes of a query's row of outputs in LDS

  // 16-byte chunks are exchanged within a row so that the fragments' reads meet no bank twice: keys are
  // read a chunk from 16 rows, values four chunks from four rows.
  __device__ static int swizzle_k(int row) { return PITCH == 256 ? row & 15 : (row >> 1) & 7; }
  __device__ static int swizzle_v(int row) { return PITCH == 256 ? 4 * (row & 3) : 4 * ((row >> 1) & 1); }

  // One pass over the keys: unnormalized O^T in acc, this lane's part of the sums in l, the (scaled) maximum in m;
  // keys kb .. ke - 1 of the sequence
  __device__ static void pass(const AttnArgs& a, const Span& s, int hk, int G, int kb, int ke, uint8_t* lds, v4u (&q)[KS],
                              v16f (&acc)[DT], float& l, float& m) {
    const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5;
    const int off = s.nk - s.nq;                                     // query i sees keys to i + off
    const int rows = s.nq * G, w0 = s.first + 32 * wid;          // the wavefront's first row
    auto sees_of = [&](int row) { return (a.causal ? min(row / G + off + 1, ke) : ke) - kb; };     // counted from kb
    const int nk = max(sees_of(min(s.first + QT, rows) - 1), 0);
    const int tiles = (nk + KT - 1) / KT;                            // that any of the workgroup's rows sees
    const int sees = sees_of(w0 + (lane & 31));                      // keys the lane's row sees
    const int wsees = w0 >= rows ? 0 : sees_of(min(w0 + 32, rows) - 1);          // any of the wavefront's
    const int wall = sees_of(w0);                                    // all of them
    const int wtiles = wsees > 0 ? (wsees + KT - 1) / KT : 0;

    const int row = ROWS * wid + lane / (PITCH / 16), ch = lane % (PITCH / 16);
    const int ck = ch ^ swizzle_k(row), cv = ch ^ swizzle_v(row), chunks = a.D / 8;
    const uint32_t vk = ck < chunks ? (uint32_t)(row * a.k.ts) + 16 * ck : (uint32_t)KQ_OOB;
    const uint32_t vv = cv < chunks ? (uint32_t)(row * a.v.ts) + 16 * cv : (uint32_t)KQ_OOB;
    const uint32_t lds0 = lds_addr(lds) + 1024 * wid;
    const uint8_t* const kp = a.k.p + (s.k0 + kb) * a.k.ts + hk * a.k.hs;
    const uint8_t* const vp = a.v.p + (s.k0 + kb) * a.v.ts + hk * a.v.hs;
    // rows behind the last key: zeros; tiles behind the last: nothing.  Tile t goes to slot t % 2.
    auto load = [&](const uint8_t* p, int64_t ts, uint32_t off, uint32_t at, int t) {
      if (t >= tiles) return;
      const v4i r = rsrc_words(p + (int64_t)KT * t * ts, (int64_t)(ke - kb - KT * t - 1) * ts + 2 * a.D);
#pragma unroll
      for (int n = 0; n < LOADS; ++n) lds_load16(r, at + 1024 * NW * n, (int)(off + (uint32_t)(ROWS * NW * n) * (uint32_t)ts));
    };
    auto load_k = [&](int t, int slot) { load(kp, a.k.ts, vk, lds0 + slot * TILE, t); };
    auto load_v = [&](int t, int slot) { load(vp, a.v.ts, vv, lds0 + (2 + slot) * TILE, t); };

    // this lane's fragment addresses within a tile
    const int kr = lane & 31;
    int ka[KS], va[DT];
#pragma unroll
    for (int i = 0; i < KS; ++i) ka[i] = PITCH * kr + 16 * ((2 * i + half) ^ swizzle_k(kr));
    const int vr = 4 * half + ((lane & 15) >> 2);                    // key of the first four
#pragma unroll
    for (int i = 0; i < DT; ++i)
      va[i] = PITCH * vr + 16 * ((4 * i + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ swizzle_v(vr)) + 8 * (lane & 1);

    float base = 0.0f;                                               // m scaled: weights are exp2(x c - base)
    v16f x[2][2];                                                    // scores of a tile, in x[t % 2]
    v4u p[4];                                                        // weights of a tile (PRECISE: they replace its scores)
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][e] = 0.0f;
    l = 0.0f;
    m = HIDDEN;

    // fragment n of a slot's keys (rows 32 (n % 2) .. + 31, contraction step n / 2) and of its values (row block n % DT,
    // contraction step n / DT)
    auto key_frag = [&](int slot, int n) {
      return *reinterpret_cast<const v4u*>(lds + slot * TILE + 32 * PITCH * (n & 1) + ka[n >> 1]);
    };
    auto value_frag = [&](int slot, int n) {
      const uint8_t* const at = lds + (2 + slot) * TILE + va[n % DT] + 16 * PITCH * (n / DT);
      const v2u lo = lds_tr16(at), hi = lds_tr16(at + 8 * PITCH);
      return v4u{lo[0], lo[1], hi[0], hi[1]};
    };
    // weights 2 n and 2 n + 1 of the lane's 32; their sum is that of the rounded ones
    auto weight_pair = [&](v16f (&y)[2], int n) {
      const int h = n >> 3, e = 2 * (n & 7);
      const float p0 = __builtin_amdgcn_exp2f(fmaf(y[h][e], a.c, -base));
      const float p1 = __builtin_amdgcn_exp2f(fmaf(y[h][e + 1], a.c, -base));
      if constexpr (PRECISE) {
        l += p0 + p1;
        y[h][e] = p0, y[h][e + 1] = p1;
      } else {
        const uint32_t w = pack2_16<BF16>(p0, p1);
        l = add_pair<BF16>(w, l);
        p[n >> 2][n & 3] = w;
      }
    };
    // the weights of contraction step k as sums of NUMBERS 16-bit numbers, the largest first
    auto split = [&](const v16f (&y)[2], int k, v4u (&w)[NUMBERS]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float p0 = y[k >> 1][8 * (k & 1) + 2 * i], p1 = y[k >> 1][8 * (k & 1) + 2 * i + 1];
#pragma unroll
        for (int u = 0; u < NUMBERS; ++u) {
          const uint32_t r = pack2_16<BF16>(p0, p1);
          w[u][i] = r;
          p0 -= unpack1_16<BF16>((uint16_t)r), p1 -= unpack1_16<BF16>((uint16_t)(r >> 16));
        }
      }
    };
    // The compiler's own order reads each fragment just before its product; these loops keep AHEAD fragments in
    // flight and put a share of the vector work behind each product.  (Heads of 128, 8192 tokens: 512, 497 and 502 us with 2,
    // 3 and 4; heads of 72 206, 207 and 205; heads of 64 leave registers for a third workgroup with 3; PRECISE spills less with
    // 2 for heads of 128.)
    constexpr int AHEAD = KS == 5 || KS == 6 ? 4 : PRECISE && KS == 8 ? 2 : 3, NK = 2 * KS, NV = 4 * DT;
    auto scores = [&](v16f (&y)[2], int slot, auto beside) {
      v4u f[NK];
      v16f z;
#pragma unroll
      for (int e = 0; e < 16; ++e) z[e] = 0.0f;
#pragma unroll
      for (int n = 0; n < AHEAD; ++n) f[n] = key_frag(slot, n);
#pragma unroll
      for (int n = 0; n < NK; ++n) {
        if (n + AHEAD < NK) f[n + AHEAD] = key_frag(slot, n + AHEAD);
        y[n & 1] = mfma32<BF16>(f[n], q[n >> 1], n < 2 ? z : y[n & 1]);
#pragma unroll
        for (int i = 16 * n / NK; i < 16 * (n + 1) / NK; ++i) beside(i);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    auto values = [&](const v16f (&y)[2], int slot, auto beside) {
      v4u f[NV], w[NUMBERS];
#pragma unroll
      for (int n = 0; n < AHEAD; ++n) f[n] = value_frag(slot, n);
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        if (n + AHEAD < NV) f[n + AHEAD] = value_frag(slot, n + AHEAD);
        if constexpr (PRECISE) {
          if (n % DT == 0) split(y, n / DT, w);
#pragma unroll
          for (int u = 0; u < NUMBERS; ++u) acc[n % DT] = mfma32<BF16>(f[n], w[u], acc[n % DT]);
        } else {
          acc[n % DT] = mfma32<BF16>(f[n], p[n / DT], acc[n % DT]);
        }
#pragma unroll
        for (int i = 16 * n / NV; i < 16 * (n + 1) / NV; ++i) beside(i);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    auto hide = [&](v16f (&y)[2], int key) {
      if (key + KT > wall) {
        const int left = sees - key - 4 * half;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            y[h][e] = 32 * h + 8 * (e >> 2) + (e & 3) < left ? y[h][e] : HIDDEN;
      }
    };
    float top;
    auto compare = [&](const v16f (&y)[2], int n) {
      top = fmaxf(fmaxf(top, y[n >> 3][2 * (n & 7)]), y[n >> 3][2 * (n & 7) + 1]);
    };
    auto raise = [&] {
      top = half_max(top) * a.c;
      if (__any(top > m + 8.0f)) {
        const float to = fmaxf(m, top);
        const float f = to == HIDDEN ? 1.0f : __builtin_amdgcn_exp2f(m - to);
        m = to;
        base = (to == HIDDEN ? 0.0f : to) - LIFT;
        l *= f;
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[i][e] *= f;
      }
    };
    // Tile t's keys one step ahead of its values: a step's products need K(t + 1) and V(t), its loads fill the slots of
    // K(t) and V(t - 1), which the step before has read.  (The first tiles' are loaded together, below.)
    auto step = [&](int t, int slot) {
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
      lds_barrier();
      load_k(t + 2, slot);
      load_v(t + 1, slot ^ 1);
    };
    // tile t, in slot S, and the scores of the next
    auto both = [&](int t, auto S) {
      constexpr int S0 = decltype(S)::value, S1 = S0 ^ 1;
      step(t, S0);
      scores(x[S1], S1, [&](int n) { weight_pair(x[S0], n); });
      if constexpr (PRECISE) asm volatile("" : "+v"(x[S0][0]), "+v"(x[S0][1]));         // here, not behind the branch
      else asm volatile("" : "+v"(p[0]), "+v"(p[1]), "+v"(p[2]), "+v"(p[3]));
      hide(x[S1], KT * (t + 1));
      top = HIDDEN;
      values(x[S0], S0, [&](int n) { compare(x[S1], n); });
      raise();
    };
    auto last = [&](int t, auto S) {
      constexpr int S0 = decltype(S)::value;
      step(t, S0);
#pragma unroll
      for (int n = 0; n < 16; ++n) weight_pair(x[S0], n);
      values(x[S0], S0, [](int) {});
    };
    const std::integral_constant<int, 0> even;
    const std::integral_constant<int, 1> odd;

    load_k(0, 0);
    load_v(0, 0);
    load_k(1, 1);
#pragma unroll
    for (int i = 0; i < KS; ++i) asm volatile("" : "+v"(q[i]));      // the queries are waited for here, not in the loop
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    lds_barrier();
    int t = 0;
    if (wtiles > 0) {
      scores(x[0], 0, [](int) {});
      hide(x[0], 0);
      top = HIDDEN;
#pragma unroll
      for (int n = 0; n < 16; ++n) compare(x[0], n);
      raise();
      for (; t + 2 < wtiles; t += 2) {
        both(t, even);
        both(t + 1, odd);
      }
      if (t + 1 < wtiles) {
        both(t++, even);
        last(t++, odd);
      } else {
        last(t++, even);
      }
    }
    for (; t < tiles; ++t) step(t, t & 1);                           // the workgroup's other wavefronts see more
  }
};

// Outputs of rows row0 .. + 31 (below `rows`): acc holds their O^T, unnormalized; `mine` is the wavefront's own LDS.
template <bool BF16, int DT, int OPITCH>
__device__ __forceinline__ void store_rows(const AttnArgs& a, const v16f (&acc)[DT], float inv, int64_t q0, int hk, int G,
                                           int row0, int rows, uint8_t* mine) {
  const int lane = threadIdx.x & 63, half = lane >> 5;
  auto place = [&](int row) { return (q0 + row / G) * a.Hq + hk * G + row % G; };      // of a row among all outputs
  if constexpr (DT == 4) {
    if (a.scales) {                                                  // D is 128
      uint32_t top = 0;
      float o[DT][16];
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          o[i][e] = acc[i][e] * inv;
          top = umax32(top, abs_bits(o[i][e]));
        }
      const auto x = __builtin_amdgcn_permlane32_swap(top, top, false, false);
      const uint32_t byte = f8_scale_byte(umax32(x[0], x[1]));
      const bool nan = byte == 255u;
      const float unit = nan ? 1.0f : f8_inv_scale(byte);
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int e = 0; e < 16; e += 4)
          *reinterpret_cast<uint32_t*>(mine + OPITCH * (lane & 31) + 32 * i + 2 * e + 4 * half) =
              nan ? 0x7F7F7F7Fu : f8_pack4(o[i][e], o[i][e + 1], o[i][e + 2], o[i][e + 3], unit);
      if (half == 0 && row0 + lane < rows) {
        const int row = row0 + lane, head = hk * G + row % G, SC = (int)f8_scale_cols((int64_t)a.Hq * 128);
        uint8_t* const at = a.scales + (q0 + row / G) * SC;
        at[head] = (uint8_t)byte;
        if (head == a.Hq - 1)
          for (int c = a.Hq; c < SC; ++c) at[c] = 0;
      }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 8 * i + (lane >> 3), c = 16 * (lane & 7);
        if (row0 + row < rows)
          *reinterpret_cast<v4u*>(static_cast<uint8_t*>(a.out) + place(row0 + row) * 128 + c) =
              *reinterpret_cast<const v4u*>(mine + OPITCH * row + c);
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int e = 0; e < 16; e += 4)
      *reinterpret_cast<v2u*>(mine + OPITCH * (lane & 31) + 64 * i + 4 * e + 8 * half) =
          v2u{pack2_16<BF16>(acc[i][e] * inv, acc[i][e + 1] * inv), pack2_16<BF16>(acc[i][e + 2] * inv, acc[i][e + 3] * inv)};
  __builtin_amdgcn_wave_barrier();
  const int chunks = a.D / 8;
  constexpr int PER = 4 * DT;                                        // chunks of a row in LDS
#pragma unroll
  for (int i = 0; i < PER / 2; ++i) {
    const int n = 64 * i + lane, row = n / PER, c = n % PER;
    if (row0 + row < rows && c < chunks)
      *reinterpret_cast<v4u*>(static_cast<uint8_t*>(a.out) + place(row0 + row) * 2 * a.D + 16 * c) =
          *reinterpret_cast<const v4u*>(mine + OPITCH * row + 16 * c);
  }
}

// Values 2 l and 2 l + 1 (l the lane) of a query's output.
template <bool BF16>
__device__ __forceinline__ void store_pair(const AttnArgs& a, int64_t token, int head, float o0, float o1) {
  const int lane = threadIdx.x & 63;
  if (a.scales) {                                                    // D is 128
    uint32_t top = row16_umax(umax32(abs_bits(o0), abs_bits(o1)));
    top = umax32(top, __shfl_xor(top, 16, 64));
    top = umax32(top, __shfl_xor(top, 32, 64));
    const uint32_t byte = f8_scale_byte(top);
    const float unit = byte == 255u ? 1.0f : f8_inv_scale(byte);
    const uint32_t w = byte == 255u ? 0x7F7Fu : f8_pack4(o0, o1, 0.0f, 0.0f, unit);
    *reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(a.out) + (token * a.Hq + head) * 128 + 2 * lane) = (uint16_t)w;
    const int SC = (int)f8_scale_cols((int64_t)a.Hq * 128);
    if (lane == 0) a.scales[token * SC + head] = (uint8_t)byte;
    if (head == a.Hq - 1 && head + 1 + lane < SC) a.scales[token * SC + head + 1 + lane] = 0;
  } else if (2 * lane < a.D) {
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.out) + ((token * a.Hq + head) * a.D + 2 * lane) * 2) =
        pack2_16<BF16>(o0, o1);
  }
}

// A row again, by the definition: a value that is not finite has reached a row that does not see it (0 times it
// is not 0), or such values are seen.  64 keys at a time: a lane has a key's score, then values 2 l and
// 2 l + 1 of the sum.  Slow (16 us for 64 keys of a row, 32 rows in turn: of 8192 tokens, 32 / 8 heads of 128, an infinite
// value at the last key takes the call from 0.5 to 67 ms, at the first 111), and small: it needs none of the tiles'
// registers.
template <bool BF16>
__device__ void exact_row(const AttnArgs& a, const Span& s, int hk, int G, int row) {
  const int lane = threadIdx.x & 63;
  const uint8_t* const kp = a.k.p + s.k0 * a.k.ts + hk * a.k.hs;
  const uint8_t* const vp = a.v.p + s.k0 * a.v.ts + hk * a.v.hs + 4 * lane;
  const int head = hk * G + row % G, n = a.causal ? min(row / G + s.nk - s.nq + 1, s.nk) : s.nk;
  const int64_t token = s.q0 + row / G;
  const uint8_t* const qp = a.q.p + token * a.q.ts + head * a.q.hs;
  float m = -INFINITY, l = 0.0f, o0 = 0.0f, o1 = 0.0f;
  for (int k0 = 0; k0 < n; k0 += 64) {
    const bool there = k0 + lane < n;
    float x = 0.0f;
    for (int c = 0; c < a.D / 8; ++c) {
      v4u kw = {0, 0, 0, 0};
      if (there) kw = *reinterpret_cast<const v4u*>(kp + (int64_t)(k0 + lane) * a.k.ts + 16 * c);
      float k[8], q[8];
      unpack8_16<BF16>(kw, k);
      unpack8_16<BF16>(*reinterpret_cast<const v4u*>(qp + 16 * c), q);
#pragma unroll
      for (int e = 0; e < 8; ++e) x = fmaf(k[e], q[e], x);
    }
    x = there ? x * a.c : -INFINITY;
    float to = fmaxf(m, x);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) to = fmaxf(to, __shfl_xor(to, off, 64));
    const float base = to == -INFINITY ? 0.0f : to, f = __builtin_amdgcn_exp2f(m - base);
    const float p = there ? __builtin_amdgcn_exp2f(x - base) : 0.0f;
    m = to;
    l = fmaf(l, f, p);
    o0 *= f, o1 *= f;
    for (int i = 0; i < min(64, n - k0); ++i) {
      const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(p), i));
      uint32_t v = 0;
      if (2 * lane < a.D) v = *reinterpret_cast<const uint32_t*>(vp + (int64_t)(k0 + i) * a.v.ts);
      o0 = fmaf(w, unpack1_16<BF16>((uint16_t)v), o0);
      o1 = fmaf(w, unpack1_16<BF16>((uint16_t)(v >> 16)), o1);
    }
  }
  // no weight at all (no key, or no score above minus infinity): zeros, whatever the values
  const float sum = wave_sum(l), inv = 1.0f / sum;
  const bool none = sum == 0.0f;
  store_pair<BF16>(a, token, head, none ? 0.0f : o0 * inv, none ? 0.0f : o1 * inv);
}

// Keys of part z of a sequence's nk, in whole tiles.
__device__ __forceinline__ int part_begin(int nk, int parts, int z) {
  const int tiles = (nk + KT - 1) / KT, per = (tiles + parts - 1) / parts;
  return (int)min((int64_t)nk, (int64_t)z * per * KT);
}

// Two workgroups on a compute unit, three or four for narrow heads (64: 4096 tokens, 32 / 8 heads, causal 100 and 92 us).  PRECISE
// keeps a tile's weights in float32, which takes one away from narrow heads; heads of 128 keep two and spill 11 to 14
// registers (one without spilling: 1072 us and not 938).
// PARTS: the keys are split, blockIdx.y says which part is the workgroup's, and what it finds goes to the workspace,
// unnormalized: values [part][token][head][32 DT], then maxima and sums of weights [part][token][head][2].
template <bool BF16, int KS, int DT, int NW, bool PARTS, bool PRECISE>
__global__ __launch_bounds__(64 * NW, KS <= 2 ? 4 - PRECISE : KS <= 4 ? 3 - PRECISE : 2) void attn_prompt_kernel(AttnArgs a, int32_t slots) {
  using P = Prompt<BF16, KS, DT, NW, PRECISE>;
  constexpr int QT = P::QT;
  constexpr int LDS = 4 * P::TILE > 32 * NW * P::OPITCH ? 4 * P::TILE : 32 * NW * P::OPITCH;
  __shared__ __align__(1024) uint8_t lds[LDS];
  // The eight compute dies take workgroups in turn.  Each is given key heads of its own (or a share of one head's
  // rows), so that its level-2 cache holds few heads' keys.  The last rows, which see the most keys, go first.
  const uint32_t id = blockIdx.x, H = a.Hkv, die = id % 8;
  uint32_t hk, slot;
  if (H % 8 == 0) {
    const uint32_t per = H / 8, i = id / 8;
    hk = die * per + i % per;
    slot = i / per;
  } else if (8 % H == 0) {
    hk = die % H;
    slot = id / 8 * (8 / H) + die / H;
    if (slot >= (uint32_t)slots) return;
  } else {
    hk = id % H;
    slot = id / H;
  }
  const int G = a.Hq / a.Hkv;
  Span s;
  if (!find_span<QT>(a, G, slots - 1 - (int32_t)slot, s)) return;

  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, w0 = s.first + 32 * wid, rows = s.nq * G;
  v4u q[KS];
  {
    const int row = w0 + (lane & 31);
    const uint8_t* const at = a.q.p + (s.q0 + row / G) * a.q.ts + (int64_t)(hk * G + row % G) * a.q.hs + 16 * half;
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      q[i] = v4u{0, 0, 0, 0};
      if (row < rows && 2 * i + half < a.D / 8) q[i] = *reinterpret_cast<const v4u*>(at + 32 * i);
    }
  }
  v16f acc[DT];
  float l;
  float m;
  const int kb = PARTS ? part_begin(s.nk, a.parts, blockIdx.y) : 0;
  P::pass(a, s, hk, G, kb, PARTS ? part_begin(s.nk, a.parts, blockIdx.y + 1) : s.nk, lds, q, acc, l, m);
  if constexpr (PARTS) {
    const float sum = half_sum(l);
    const int row = w0 + (lane & 31);
    if (row >= rows) return;
    const int64_t R = a.T * a.Hq, at = blockIdx.y * R + (s.q0 + row / G) * a.Hq + hk * G + row % G;
    if (half == 0) {
      float* const ml = a.part + a.parts * R * 32 * DT + 2 * at;
      ml[0] = m, ml[1] = sum;
    }
    float* const o = a.part + at * 32 * DT + 4 * half;
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        *reinterpret_cast<v4f*>(o + 32 * i + 2 * e) = v4f{acc[i][e], acc[i][e + 1], acc[i][e + 2], acc[i][e + 3]};
    return;
  }
  lds_barrier();                                                     // the tiles have been read: outputs go there
  float zero = 0.0f;
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) zero = fmaf(acc[i][e], 0.0f, zero);
  if (__builtin_expect(__any(!(zero == 0.0f)), 0)) {
    for (int row = w0; row < min(w0 + 32, rows); ++row) exact_row<BF16>(a, s, hk, G, row);
    return;
  }
  const float sum = half_sum(l), inv = sum == 0.0f ? 0.0f : 1.0f / sum;        // a query that sees nothing: zeros
  store_rows<BF16, DT, P::OPITCH>(a, acc, inv, s.q0, hk, G, w0, rows, lds + 32 * P::OPITCH * wid);
}

// Joins the parts of a row, one wavefront each: lane l has part l's maximum and sum, then values 2 l and 2 l + 1.
template <bool BF16, int DT>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t R = a.T * a.Hq, at = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (at >= R) return;
  const int head = (int)(at % a.Hq), G = a.Hq / a.Hkv, hk = head / G;
  const int32_t token = (int32_t)(at / a.Hq);
  // the token's sequence: the last that begins up to it
  Span s = {0, 0, (int32_t)a.T, (int32_t)a.Tk, 0};
  if (a.cu_q) {
    const int32_t T = (int32_t)a.T, Tk = (int32_t)a.Tk;
    const int i = last_before(a.B, [&](int i) { return a.cu_q[i] <= token; });
    const int32_t q0 = min(max(a.cu_q[i], 0), T), q1 = min(max(a.cu_q[i + 1], q0), T);
    const int32_t k0 = min(max(a.cu_k[i], 0), Tk), k1 = min(max(a.cu_k[i + 1], k0), Tk);
    if (token < q0 || token >= q1) return;
    s = {q0, k0, q1 - q0, k1 - k0, 0};
  }
  float m = -INFINITY, l = 0.0f;
  if (lane < a.parts) {
    const float* const ml = a.part + a.parts * R * 32 * DT + 2 * (lane * R + at);
    m = ml[0], l = ml[1];
  }
  float top = m;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
  const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - top);
  const float sum = wave_sum(lane < a.parts ? f * l : 0.0f);
  // Parts that begin behind the last key that the row sees are left out, whatever those keys' values have made of their
  // sums.  The others count even if their weights vanish (or are none) beside another part's, so that what is not finite
  // among them is looked at again below.
  const int32_t row = (token - (int32_t)s.q0) * G + head % G;
  const int32_t sees = a.causal ? min(row / G + s.nk - s.nq + 1, s.nk) : s.nk;
  const uint64_t unseen = __ballot(lane < a.parts && part_begin(s.nk, a.parts, lane) >= sees);
  float o0 = 0.0f, o1 = 0.0f;
  if (2 * lane < 32 * DT) {
    const float* const o = a.part + at * 32 * DT + 2 * lane;
#pragma unroll 4
    for (int z = 0; z < a.parts; ++z) {
      const float2 v = *reinterpret_cast<const float2*>(o + z * R * 32 * DT);
      const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), z));
      const bool skip = unseen >> z & 1;
      o0 = skip ? o0 : fmaf(w, v.x, o0);
      o1 = skip ? o1 : fmaf(w, v.y, o1);
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  o0 *= inv, o1 *= inv;
  if (__builtin_expect(__any(!(fabsf(o0) < INFINITY && fabsf(o1) < INFINITY)), 0))
    exact_row<BF16>(a, s, hk, G, row);
  else
    store_pair<BF16>(a, token, head, o0, o1);
}

constexpr int NW = 4, QT = 32 * NW;

int64_t slots_of(int64_t T, int64_t B, bool packed, int G) { return packed ? T * G / QT + B : (T * G + QT - 1) / QT; }

// Parts that the keys are split into where there are few rows: as many as give each compute unit a workgroup (or, of very
// many tiles, two), of four tiles at least, if they save more tiles' time (0.9 us) than the joining costs, which is a
// launch and the parts' bytes.  Causal, 32 / 8 heads of 128 in bf16, whole and split (us): 16 queries of 1024 keys 22 and 14,
// of 4096 65 and 16; 256 of 2048 38 and 24; 700 of 16384 247 and 216, of 1024 24 and (not done) 30.
// Up to 704 keys (11 tiles, of which two parts save five) are never split: kq.h says so, and callers spare themselves the
// question.
int parts_of(int64_t T, int64_t Tk, int64_t B, bool packed, int Hq, int Hkv) {
  if (Tk <= 704) return 1;
  const int64_t groups = slots_of(T, B, packed, Hq / Hkv) * Hkv, tiles = (Tk + KT - 1) / KT, cus = device_cu_count();
  int64_t parts = cus / groups;
  if (parts < 2 && tiles >= 128) parts = 2 * cus / groups;
  parts = parts < tiles / 4 ? parts : tiles / 4;
  parts = parts < 64 ? parts : 64;
  if (parts < 2) return 1;
  return tiles - (tiles + parts - 1) / parts >= 6 + T * Hq * parts / 8192 ? (int)parts : 1;
}

template <bool BF16, int KS, int DT, bool PRECISE>
hipError_t go(const AttnArgs& a, hipStream_t s) {
  const int64_t slots = slots_of(a.T, a.B, a.cu_q != nullptr, a.Hq / a.Hkv);
  const int64_t grid = a.Hkv % 8 && 8 % a.Hkv == 0 ? (slots + 8 / a.Hkv - 1) / (8 / a.Hkv) * 8 : slots * a.Hkv;
  if (a.parts == 1) {
    hipLaunchKernelGGL((attn_prompt_kernel<BF16, KS, DT, NW, false, PRECISE>), dim3((unsigned)grid), dim3(64 * NW), 0, s, a,
                       (int32_t)slots);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((attn_prompt_kernel<BF16, KS, DT, NW, true, PRECISE>), dim3((unsigned)grid, (unsigned)a.parts), dim3(64 * NW), 0, s,
                     a, (int32_t)slots);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attn_join_kernel<BF16, DT>), dim3((unsigned)((a.T * a.Hq + 3) / 4)), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <bool BF16, bool PRECISE>
hipError_t by_width(const AttnArgs& a, hipStream_t s) {
  if (a.D <= 32) return go<BF16, 2, 1, PRECISE>(a, s);
  if (a.D <= 64) return go<BF16, 4, 2, PRECISE>(a, s);
  if (a.D <= 80) return go<BF16, 5, 3, PRECISE>(a, s);
  if (a.D <= 96) return go<BF16, 6, 3, PRECISE>(a, s);
  return go<BF16, 8, 4, PRECISE>(a, s);
}

}  // namespace

size_t attention_workspace_bytes(int64_t B, int64_t T, int64_t Tk, bool packed, int Hq, int Hkv, int D) {
  const int parts = parts_of(T, Tk, B, packed, Hq, Hkv);
  return parts == 1 ? 0 : (size_t)parts * T * Hq * ((D + 31) / 32 * 32 + 2) * sizeof(float);
}

hipError_t launch_attention(bool bf16, bool precise, const AttnArgs& args, hipStream_t s) {
  AttnArgs a = args;
  a.parts = parts_of(a.T, a.Tk, a.B, a.cu_q != nullptr, a.Hq, a.Hkv);
  if (precise) return bf16 ? by_width<true, true>(a, s) : by_width<false, true>(a, s);
  return bf16 ? by_width<true, false>(a, s) : by_width<false, false>(a, s);
}

}  // namespace kq
