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
// float32 sums or 16-bit weights), which spares most rescalings of the 16 DT accumulators.
#include "kq_attn.hpp"
#include "kq_launch.hpp"

namespace kq {

namespace {

constexpr int KT = 64;                 // keys of a tile

// Where a workgroup's queries and keys are.
struct Span {
  int64_t q0, k0;                      // first query of the sequence, first key
  int32_t nq, nk;                      // their numbers
  int32_t first;                       // the workgroup's first query within the sequence
};

// Sequence i's queries begin at slot cu_q[i] / QT + i of the grid, which leaves each at least as many
// slots as it has tiles without anyone having summed the tiles: a slot finds its sequence by counting
// the starts up to itself, 64 at a time.  Entries are held to 0 .. T and to their order.
template <int QT>
__device__ bool find_span(const AttnArgs& a, int32_t slot, Span& s) {
  if (!a.cu_q) {
    s = {0, 0, (int32_t)a.T, (int32_t)a.Tk, slot * QT};
    return true;
  }
  const int lane = threadIdx.x & 63;
  const int32_t T = (int32_t)a.T, Tk = (int32_t)a.Tk;
  int n = 0;
  for (int i0 = 0; i0 < a.B; i0 += 64) {
    const int i = i0 + lane;
    const bool before = i < a.B && min(max(a.cu_q[i], 0), T) / QT + i <= slot;
    const int c = __popcll(__ballot(before));
    n += c;
    if (c < 64) break;
  }
  const int i = __builtin_amdgcn_readfirstlane(max(n - 1, 0));
  const int32_t q0 = min(max(a.cu_q[i], 0), T), q1 = min(max(a.cu_q[i + 1], q0), T);
  const int32_t k0 = min(max(a.cu_k[i], 0), Tk), k1 = min(max(a.cu_k[i + 1], k0), Tk);
  s = {q0, k0, q1 - q0, k1 - k0, (slot - (q0 / QT + i)) * QT};
  return s.first >= 0 && s.first < s.nq;                   // entries out of order lead to no slot below 0
}

// Scores of masked keys.
constexpr float HIDDEN = -INFINITY;

template <bool BF16, int KS, int DT, int NW>
struct Prompt {
  static constexpr int QT = 32 * NW;
  static constexpr int PITCH = KS <= 4 ? 128 : 256;                  // bytes of a key's row in LDS
  static constexpr int TILE = KT * PITCH;
  static constexpr int LOADS = TILE / (1024 * NW);                   // of a wavefront, a matrix and tile
  static constexpr int ROWS = 1024 / PITCH;                          // rows of a load
  static constexpr int OPITCH = 64 * DT + 16;                        // bytes of a query's row of outputs in LDS

  // 16-byte chunks are exchanged within a row so that the fragments' reads meet no bank twice: keys are
  // read a chunk from 16 rows, values four chunks from four rows.
  __device__ static int swizzle_k(int row) { return PITCH == 256 ? row & 15 : (row >> 1) & 7; }
  __device__ static int swizzle_v(int row) { return PITCH == 256 ? 4 * (row & 3) : 4 * ((row >> 1) & 1); }

  // One pass over the keys: unnormalized O^T in acc, this lane's part of the sums in l.  SAFE: infinities
  // and NaN among the values reach only the queries that see them (0 times either would not be 0).
  template <bool SAFE>
  __device__ static void pass(const AttnArgs& a, const Span& s, int head, uint8_t* lds, const v4u (&q)[KS], v16f (&acc)[DT],
                              float& l) {
    const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, hk = head / (a.Hq / a.Hkv);
    const int off = s.nk - s.nq;                                     // query i sees keys to i + off
    const int last = min(s.first + QT, s.nq) - 1;
    const int nk = a.causal ? max(min(s.nk, last + off + 1), 0) : s.nk;
    const int tiles = (nk + KT - 1) / KT;
    const int mine = s.first + 32 * wid + (lane & 31);               // this lane's query
    const int sees = a.causal ? min(mine + off + 1, s.nk) : s.nk;    // keys it sees
    const int w0 = s.first + 32 * wid;
    const int wsees = w0 >= s.nq ? 0 : a.causal ? min(w0 + 32 + off, s.nk) : s.nk;   // any of the wavefront's
    const int wall = a.causal ? min(w0 + off + 1, s.nk) : s.nk;      // all of them

    const int row = ROWS * wid + lane / (PITCH / 16), ch = lane % (PITCH / 16);
    const int ck = ch ^ swizzle_k(row), cv = ch ^ swizzle_v(row), chunks = a.D / 8;
    const uint32_t vk = ck < chunks ? (uint32_t)(row * a.k.ts) + 16 * ck : (uint32_t)KQ_OOB;
    const uint32_t vv = cv < chunks ? (uint32_t)(row * a.v.ts) + 16 * cv : (uint32_t)KQ_OOB;
    const uint32_t lds0 = lds_addr(lds) + 1024 * wid;
    const uint8_t* const kp = a.k.p + s.k0 * a.k.ts + hk * a.k.hs;
    const uint8_t* const vp = a.v.p + s.k0 * a.v.ts + hk * a.v.hs;
    auto load = [&](int t) {
      const int left = s.nk - KT * t;                                // rows behind the last key: zeros
      const v4i rk = rsrc_words(kp + (int64_t)KT * t * a.k.ts, (int64_t)(left - 1) * a.k.ts + 2 * a.D);
      const v4i rv = rsrc_words(vp + (int64_t)KT * t * a.v.ts, (int64_t)(left - 1) * a.v.ts + 2 * a.D);
      const uint32_t at = lds0 + (t & 1) * 2 * TILE;
#pragma unroll
      for (int n = 0; n < LOADS; ++n) lds_load16(rk, at + 1024 * NW * n, (int)(vk + (uint32_t)(ROWS * NW * n) * (uint32_t)a.k.ts));
#pragma unroll
      for (int n = 0; n < LOADS; ++n)
        lds_load16(rv, at + TILE + 1024 * NW * n, (int)(vv + (uint32_t)(ROWS * NW * n) * (uint32_t)a.v.ts));
    };

    // this lane's fragment addresses within a tile
    const int kr = lane & 31;
    int ka[KS], va[DT];
#pragma unroll
    for (int i = 0; i < KS; ++i) ka[i] = PITCH * kr + 16 * ((2 * i + half) ^ swizzle_k(kr));
    const int vr = 4 * half + ((lane & 15) >> 2);                    // key of the first four
#pragma unroll
    for (int i = 0; i < DT; ++i)
      va[i] = PITCH * vr + 16 * ((4 * i + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ swizzle_v(vr)) + 8 * (lane & 1);

#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][e] = 0.0f;
    l = 0.0f;
    float m = HIDDEN;                                                // scaled: exponents are x c - m
    if (tiles > 0) load(0);
    for (int t = 0; t < tiles; ++t) {
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
      lds_barrier();
      if (t + 1 < tiles) load(t + 1);
      const int key = KT * t;
      if (key >= wsees) continue;                                    // nothing here that this wavefront sees
      const uint8_t* const tk = lds + (t & 1) * 2 * TILE;
      const uint8_t* const tv = tk + TILE;
      v16f x[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[h][e] = 0.0f;
#pragma unroll
        for (int i = 0; i < KS; ++i)
          x[h] = mfma32<BF16>(*reinterpret_cast<const v4u*>(tk + 32 * PITCH * h + ka[i]), q[i], x[h]);
      }
      if (key + KT > wall) {
        const int left = sees - key - 4 * half;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            x[h][e] = 32 * h + 8 * (e >> 2) + (e & 3) < left ? x[h][e] : HIDDEN;
      }
      float top = HIDDEN;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, x[h][e]);
      top = half_max(top) * a.c;
      if (__any(top > m + 8.0f)) {
        const float to = fmaxf(m, top);
        const float f = to == HIDDEN ? 1.0f : __builtin_amdgcn_exp2f(m - to);
        m = to;
        l *= f;
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[i][e] *= f;
      }
      const float base = m == HIDDEN ? 0.0f : m;
      float sum = 0.0f;
      v4u p[4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const float p0 = __builtin_amdgcn_exp2f(fmaf(x[h][e], a.c, -base));
          const float p1 = __builtin_amdgcn_exp2f(fmaf(x[h][e + 1], a.c, -base));
          sum += p0 + p1;
          p[2 * h + (e >> 3)][(e & 7) >> 1] = pack2_16<BF16>(p0, p1);
        }
      l += sum;
#pragma unroll
      for (int i = 0; i < DT; ++i) {
        if constexpr (SAFE) {
          v16f up, down;
#pragma unroll
          for (int e = 0; e < 16; ++e) up[e] = down[e] = 0.0f;
          constexpr uint32_t INF = BF16 ? 0x7F80u : 0x7C00u, ONE = BF16 ? 0x3F80u : 0x3C00u;
          for (int j = 0; j < 4; ++j) {
            const uint8_t* const at = tv + va[i] + 16 * PITCH * j;
            const v2u lo = lds_tr16(at), hi = lds_tr16(at + 8 * PITCH);
            const v4u b = j == 0 ? p[0] : j == 1 ? p[1] : j == 2 ? p[2] : p[3];
            v4u fin = {lo[0], lo[1], hi[0], hi[1]}, pos = {0, 0, 0, 0}, neg = {0, 0, 0, 0}, see = {0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int sh = 16 * (e & 1);
              const uint32_t w = (fin[e / 2] >> sh) & 0xFFFFu;
              if ((w & INF) == INF) {
                fin[e / 2] &= ~(0xFFFFu << sh);
                if (w != (INF | 0x8000u)) pos[e / 2] |= ONE << sh;
                if (w != INF) neg[e / 2] |= ONE << sh;
              }
              if (key + 16 * j + 8 * (e >> 2) + 4 * half + (e & 3) < sees) see[e / 2] |= ONE << sh;
            }
            acc[i] = mfma32<BF16>(fin, b, acc[i]);
            up = mfma32<BF16>(pos, see, up);
            down = mfma32<BF16>(neg, see, down);
          }
#pragma unroll
          for (int e = 0; e < 16; ++e)
            acc[i][e] += (up[e] > 0.0f ? INFINITY : 0.0f) + (down[e] > 0.0f ? -INFINITY : 0.0f);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint8_t* const at = tv + va[i] + 16 * PITCH * j;
            const v2u lo = lds_tr16(at), hi = lds_tr16(at + 8 * PITCH);
            acc[i] = mfma32<BF16>(v4u{lo[0], lo[1], hi[0], hi[1]}, p[j], acc[i]);
          }
        }
      }
    }
  }
};

template <bool BF16, int KS, int DT, int NW>
__global__ __launch_bounds__(64 * NW) void attn_prompt_kernel(AttnArgs a, int32_t slots) {
  using P = Prompt<BF16, KS, DT, NW>;
  constexpr int QT = P::QT;
  constexpr int LDS = 4 * P::TILE > 32 * NW * P::OPITCH ? 4 * P::TILE : 32 * NW * P::OPITCH;
  __shared__ __align__(1024) uint8_t lds[LDS];
  // The compute dies take workgroups in turn; each is given heads of its own (the queries' heads of one
  // key head next to each other), so that a die's level-2 cache holds few heads' keys.  The last queries,
  // who see the most keys, go first.
  const uint32_t id = blockIdx.x, H = a.Hq;
  uint32_t head, slot;
  if (H % 8 == 0) {
    const uint32_t per = H / 8, i = id / 8;
    head = id % 8 * per + i % per;
    slot = i / per;
  } else {
    head = id % H;
    slot = id / H;
  }
  Span s;
  if (!find_span<QT>(a, slots - 1 - (int32_t)slot, s)) return;

  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, w0 = s.first + 32 * wid, rows = min(32, s.nq - w0);
  v4u q[KS];
  {
    const __amdgpu_buffer_rsrc_t rq =
        make_rsrc(a.q.p + (s.q0 + w0) * a.q.ts + head * a.q.hs, rows > 0 ? (rows - 1) * a.q.ts + 2 * a.D : 0);
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      const int ch = 2 * i + half;
      const int at = ch < a.D / 8 ? (lane & 31) * (int)a.q.ts + 16 * ch : KQ_OOB;
      q[i] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(rq, at, 0, 0));
    }
#pragma unroll
    for (int i = 0; i < KS; ++i) asm volatile("" : "+v"(q[i]));      // here before the loop's own loads
  }
  v16f acc[DT];
  float l;
  P::template pass<false>(a, s, head, lds, q, acc, l);
  l = half_sum(l);
  bool bad = false;
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) bad |= !(fabsf(acc[i][e]) < INFINITY);
  if (__builtin_expect(__syncthreads_or(bad), 0)) {                  // rare: the pass again, with care
    P::template pass<true>(a, s, head, lds, q, acc, l);
    l = half_sum(l);
    __syncthreads();
  }
  const float r = l == 0.0f ? 0.0f : 1.0f / l;                       // a query that sees nothing: zeros
  const int64_t t0 = s.q0 + w0;

  // whole rows through LDS
  uint8_t* const mine = lds + 32 * P::OPITCH * wid;
  if constexpr (DT == 4 && KS == 8) {
    if (a.scales) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          acc[i][e] *= r;
          top = umax32(top, abs_bits(acc[i][e]));
        }
      const auto o = __builtin_amdgcn_permlane32_swap(top, top, false, false);
      const uint32_t byte = f8_scale_byte(umax32(o[0], o[1]));
      const bool nan = byte == 255u;
      const float inv = nan ? 1.0f : f8_inv_scale(byte);
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int e = 0; e < 16; e += 4)
          *reinterpret_cast<uint32_t*>(mine + P::OPITCH * (lane & 31) + 32 * i + 2 * e + 4 * half) =
              nan ? 0x7F7F7F7Fu : f8_pack4(acc[i][e], acc[i][e + 1], acc[i][e + 2], acc[i][e + 3], inv);
      const int64_t SC = f8_scale_cols((int64_t)a.Hq * 128);
      if (half == 0 && lane < rows) {
        uint8_t* const at = a.scales + (t0 + lane) * SC;
        at[head] = (uint8_t)byte;
        if (head == H - 1)
          for (int64_t c = H; c < SC; ++c) at[c] = 0;
      }
      __builtin_amdgcn_wave_barrier();
      uint8_t* const out = static_cast<uint8_t*>(a.out) + (t0 * a.Hq + head) * 128;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 8 * i + (lane >> 3), c = 16 * (lane & 7);
        if (row < rows)
          *reinterpret_cast<v4u*>(out + (int64_t)row * a.Hq * 128 + c) = *reinterpret_cast<const v4u*>(mine + P::OPITCH * row + c);
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int e = 0; e < 16; e += 4)
      *reinterpret_cast<v2u*>(mine + P::OPITCH * (lane & 31) + 64 * i + 4 * e + 8 * half) =
          v2u{pack2_16<BF16>(acc[i][e] * r, acc[i][e + 1] * r), pack2_16<BF16>(acc[i][e + 2] * r, acc[i][e + 3] * r)};
  __builtin_amdgcn_wave_barrier();
  uint8_t* const out = static_cast<uint8_t*>(a.out) + (t0 * a.Hq + head) * 2 * a.D;
  const int chunks = a.D / 8;
  constexpr int PER = 4 * DT;                                        // chunks of a row in LDS
#pragma unroll
  for (int i = 0; i < PER / 2; ++i) {
    const int n = 64 * i + lane, row = n / PER, c = n % PER;
    if (row < rows && c < chunks)
      *reinterpret_cast<v4u*>(out + (int64_t)row * a.Hq * 2 * a.D + 16 * c) =
          *reinterpret_cast<const v4u*>(mine + P::OPITCH * row + 16 * c);
  }
}

template <bool BF16, int KS, int DT>
hipError_t go(const AttnArgs& a, hipStream_t s) {
  constexpr int NW = 4, QT = 32 * NW;
  const int64_t slots = a.cu_q ? a.T / QT + a.B : (a.T + QT - 1) / QT;
  hipLaunchKernelGGL((attn_prompt_kernel<BF16, KS, DT, NW>), dim3((unsigned)(slots * a.Hq)), dim3(64 * NW), 0, s, a,
                     (int32_t)slots);
  return hipGetLastError();
}

template <bool BF16>
hipError_t by_width(const AttnArgs& a, hipStream_t s) {
  if (a.D <= 32) return go<BF16, 2, 1>(a, s);
  if (a.D <= 64) return go<BF16, 4, 2>(a, s);
  if (a.D <= 80) return go<BF16, 5, 3>(a, s);
  if (a.D <= 96) return go<BF16, 6, 3>(a, s);
  return go<BF16, 8, 4>(a, s);
}

}  // namespace

hipError_t launch_attention(bool bf16, const AttnArgs& a, hipStream_t s) {
  return bf16 ? by_width<true>(a, s) : by_width<false>(a, s);
}

}  // namespace kq
