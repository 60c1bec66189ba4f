// C ABI of the 8-bit path's attention: host-side argument validation and dispatch to the kernels.
#include <cmath>

#include "kq.h"
#include "kq_attn.hpp"

using namespace kq;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

kq_status hip_status(hipError_t e) { return e == hipSuccess ? KQ_OK : KQ_ERR_HIP; }

kq_status check_heads(int32_t dtype, int32_t Hq, int32_t Hkv, int32_t D, bool wide) {
  if (dtype != KQ_DT_F16 && dtype != KQ_DT_BF16) return KQ_ERR_UNSUPPORTED;
  if (Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || D < 8 || D % (wide ? 8 : 16) != 0) return KQ_ERR_SHAPE;
  if (D > 128 || Hq > 4096) return KQ_ERR_UNSUPPORTED;
  return KQ_OK;
}

// Strides in elements: whole 16-byte pieces, rows that do not overlap, 32-bit offsets over a tile's rows.
kq_status check_rows(const void* p, int64_t token, int64_t head, int32_t D, int64_t head_most) {
  if (!aligned(p, 16)) return KQ_ERR_ALIGN;
  if (token % 8 != 0 || head % 8 != 0 || token < D || head < 0) return KQ_ERR_SHAPE;
  if (token > (1LL << 21) || head > head_most) return KQ_ERR_UNSUPPORTED;
  return KQ_OK;
}

kq_status check_output(const void* O, const uint8_t* codes, const uint8_t* scales, int32_t D) {
  if (O ? codes || scales : !codes || !scales) return KQ_ERR_NULL;
  if (!O && D != 128) return KQ_ERR_UNSUPPORTED;
  if (!aligned(O, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return KQ_ERR_ALIGN;
  return KQ_OK;
}

kq_status check_cache(const void* kc, const void* vc, const uint8_t* ks, const uint8_t* vs, int64_t pages, int32_t page,
                      const int32_t* table, int64_t width, const int32_t* lengths, int64_t B) {
  if (!kc || !vc || !table || !lengths || !ks != !vs) return KQ_ERR_NULL;
  if (B < 1 || pages < 1 || width < 1 || page < 16 || page % 16 != 0) return KQ_ERR_SHAPE;
  if (B > (1LL << 20) || pages > 0x7FFFFFFFLL || page > 65536 || width > (1LL << 30) / page ||
      B > (1LL << 37) / (width * page))
    return KQ_ERR_UNSUPPORTED;
  if (!aligned(kc, 16) || !aligned(vc, 16) || !aligned(ks, 16) || !aligned(vs, 16) || !aligned(table, 4) ||
      !aligned(lengths, 4))
    return KQ_ERR_ALIGN;
  return KQ_OK;
}

kq_status check_sizes(int64_t B, int64_t T, int64_t Tk, int32_t Hq) {
  if (T < 1 || Tk < 1 || B < 1) return KQ_ERR_SHAPE;
  if (T > (1LL << 30) || Tk > (1LL << 30) || T > (1LL << 29) / Hq || B > (1LL << 22) / Hq) return KQ_ERR_UNSUPPORTED;
  return KQ_OK;
}

AttnRows rows_of(const void* p, int64_t token, int64_t head) {
  return {static_cast<const uint8_t*>(p), 2 * token, 2 * head};
}

constexpr float LOG2E = 1.4426950408889634f;

}  // namespace

extern "C" {

size_t kq_attention_workspace_bytes(int64_t B, int64_t T, int64_t Tk, int32_t packed, int32_t Hq, int32_t Hkv, int32_t D) {
  if (check_heads(KQ_DT_F16, Hq, Hkv, D, true) != KQ_OK || check_sizes(B, T, Tk, Hq) != KQ_OK) return 0;
  return attention_workspace_bytes(B, T, Tk, packed != 0, Hq, Hkv, D);
}

kq_status kq_attention(int32_t dtype, const void* Q, int64_t q_token, int64_t q_head, const void* K, int64_t k_token,
                       int64_t k_head, const void* V, int64_t v_token, int64_t v_head, const int32_t* cu_q,
                       const int32_t* cu_k, int64_t B, int64_t T, int64_t Tk, int32_t Hq, int32_t Hkv, int32_t D,
                       int32_t causal, float scale, void* O, uint8_t* codes, uint8_t* scales, void* workspace,
                       size_t workspace_bytes, hipStream_t stream) {
  const bool precise = (dtype & KQ_FP8_PRECISE) != 0;
  dtype &= ~KQ_FP8_PRECISE;
  if (!Q || !K || !V || !cu_q != !cu_k) return KQ_ERR_NULL;
  kq_status st = check_heads(dtype, Hq, Hkv, D, true);
  if (st == KQ_OK) st = check_output(O, codes, scales, D);
  if (st != KQ_OK) return st;
  st = check_sizes(B, T, Tk, Hq);
  if (st != KQ_OK) return st;
  if (!cu_q && B != 1) return KQ_ERR_SHAPE;
  st = check_rows(Q, q_token, q_head, D, 1LL << 40);
  if (st == KQ_OK) st = check_rows(K, k_token, k_head, D, 1LL << 40);
  if (st == KQ_OK) st = check_rows(V, v_token, v_head, D, 1LL << 40);
  if (st != KQ_OK) return st;
  if (!aligned(cu_q, 4) || !aligned(cu_k, 4)) return KQ_ERR_ALIGN;
  if (!std::isfinite(scale) || !(scale > 0.0f) || !std::isfinite(scale * LOG2E)) return KQ_ERR_VALUE;
  const size_t need = attention_workspace_bytes(B, T, Tk, cu_q != nullptr, Hq, Hkv, D);
  if (need && (!workspace || workspace_bytes < need)) return KQ_ERR_WORKSPACE;
  if (need && !aligned(workspace, 256)) return KQ_ERR_ALIGN;
  AttnArgs a;
  a.part = static_cast<float*>(workspace);
  a.q = rows_of(Q, q_token, q_head);
  a.k = rows_of(K, k_token, k_head);
  a.v = rows_of(V, v_token, v_head);
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.T = T;
  a.Tk = Tk;
  a.B = (int32_t)B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.causal = causal != 0;
  a.c = scale * LOG2E;
  a.out = O ? O : codes;
  a.scales = scales;
  return hip_status(launch_attention(dtype == KQ_DT_BF16, precise, a, stream));
}

kq_status kq_cache_append(int32_t dtype, const void* K, int64_t k_token, int64_t k_head, const void* V, int64_t v_token,
                          int64_t v_head, const int32_t* cu, int64_t B, int64_t T, int32_t Hkv, int32_t D,
                          const int32_t* table, int64_t width, const int32_t* lengths, void* kcache, void* vcache,
                          uint8_t* kscales, uint8_t* vscales, int64_t pages, int32_t page, hipStream_t stream) {
  if (!K || !V) return KQ_ERR_NULL;
  kq_status st = check_heads(dtype, Hkv, Hkv, D, !kscales);
  if (st == KQ_OK) st = check_cache(kcache, vcache, kscales, vscales, pages, page, table, width, lengths, B);
  if (st != KQ_OK) return st;
  if (T < 1 || (!cu && T != B)) return KQ_ERR_SHAPE;
  if (T > (1LL << 25)) return KQ_ERR_UNSUPPORTED;            // a launch is at most 2^32 threads
  st = check_rows(K, k_token, k_head, D, 1LL << 40);
  if (st == KQ_OK) st = check_rows(V, v_token, v_head, D, 1LL << 40);
  if (st != KQ_OK) return st;
  if (!aligned(cu, 4)) return KQ_ERR_ALIGN;
  AppendArgs a;
  a.c = {static_cast<uint8_t*>(kcache), static_cast<uint8_t*>(vcache), kscales, vscales, table, lengths, pages,
         (int32_t)B, (int32_t)width, page, Hkv, D};
  a.k = rows_of(K, k_token, k_head);
  a.v = rows_of(V, v_token, v_head);
  a.cu = cu;
  a.T = T;
  return hip_status(launch_cache_append(dtype == KQ_DT_BF16, !kscales, a, stream));
}

size_t kq_paged_attention_workspace_bytes(int64_t B, int32_t Hq, int32_t Hkv, int32_t D, int64_t width, int32_t page) {
  if (check_heads(KQ_DT_F16, Hq, Hkv, D, true) != KQ_OK || B < 1 || width < 1 || page < 16 || page % 16 != 0) return 0;
  if (B > (1LL << 23) / Hq || B > (1LL << 20) || page > 65536 || width > (1LL << 30) / page ||
      B > (1LL << 37) / (width * page))
    return 0;
  return paged_workspace_bytes(B, Hq, Hkv, D, width * page);
}

kq_status kq_paged_attention(int32_t dtype, const void* Q, int64_t q_seq, int64_t q_head, const void* kcache,
                             const void* vcache, const uint8_t* kscales, const uint8_t* vscales, int64_t pages,
                             int32_t page, const int32_t* table, int64_t width, const int32_t* lengths, int64_t B,
                             int32_t Hq, int32_t Hkv, int32_t D, float scale, void* O, uint8_t* codes, uint8_t* scales,
                             void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!Q) return KQ_ERR_NULL;
  kq_status st = check_heads(dtype, Hq, Hkv, D, !kscales);
  if (st == KQ_OK) st = check_output(O, codes, scales, D);
  if (st == KQ_OK) st = check_cache(kcache, vcache, kscales, vscales, pages, page, table, width, lengths, B);
  if (st != KQ_OK) return st;
  if (B > (1LL << 23) / Hq) return KQ_ERR_UNSUPPORTED;
  st = check_rows(Q, q_seq, q_head, D, 1LL << 21);
  if (st != KQ_OK) return st;
  if (!std::isfinite(scale) || !(scale > 0.0f) || !std::isfinite(scale * LOG2E)) return KQ_ERR_VALUE;
  const size_t need = paged_workspace_bytes(B, Hq, Hkv, D, width * page);
  if (need && (!workspace || workspace_bytes < need)) return KQ_ERR_WORKSPACE;
  if (need && !aligned(workspace, 256)) return KQ_ERR_ALIGN;
  PagedArgs a;
  a.c = {static_cast<uint8_t*>(const_cast<void*>(kcache)), static_cast<uint8_t*>(const_cast<void*>(vcache)),
         const_cast<uint8_t*>(kscales), const_cast<uint8_t*>(vscales), table, lengths, pages, (int32_t)B, (int32_t)width,
         page, Hkv, D};
  a.q = static_cast<const uint8_t*>(Q);
  a.qs = 2 * q_seq;
  a.qh = 2 * q_head;
  a.Hq = Hq;
  a.scale = scale * LOG2E;
  a.out = O ? O : codes;
  a.scales = scales;
  a.part = static_cast<float*>(workspace);
  return hip_status(launch_paged_attention(dtype == KQ_DT_BF16, !kscales, a, stream));
}

}  // extern "C"
