/*
 * kq — the online 4-bit activation path of a quantized diffusion-transformer linear
 * layer, for AMD Instinct MI355X (gfx950).  C ABI.
 *
 * The method (from the pages this library implements):
 *   - KroQuant (Kronecker-Structured Block Transforms for Efficient Post-Training
 *     Quantization of Diffusion Transformers), §01: Y = (XP)(P^-1 W) — an invertible
 *     transform P applied to the activations online, its inverse folded into the
 *     weights offline; §02: P = A (x) B (A 4x4, B 8x8) on every 32-element block of
 *     the activation vector; §03: 4-bit MXFP4 target format.
 *   - OrbitQuant (data-independent quantization for image and video DiTs), §03:
 *     RPBH(X) = X.P.H.D (random permutation, block Hadamard, random signs), the
 *     inverse folded offline as W' = R^-1 W, one Lloyd-Max codebook for all
 *     rotated coordinates.
 *   - CentriQ (Calibration-Free Quantization of DiTs via Exact Mean Centering),
 *     arXiv abstract: tokens are centred before the rotation and their means come
 *     back as a rank-1 fp16 term mu wbar^T; the per-token scale has a closed form.
 *   - SVDQuant explainer, §3: a 16-bit low-rank branch L1 L2 added to the 4-bit
 *     product, fused into the 4-bit kernel so it costs no separate pass; the branch
 *     holds the weight's leading singular directions, the residual is quantized.
 *   - DMQ explainer: channel-wise power-of-two scaling of outlier channels, a bit
 *     shift, as an optional step ahead of the transform.
 *
 * Layouts (all row-major, contiguous, device memory unless stated):
 *   X     fp16 [M][K]           activations, K a multiple of 32
 *   codes u8   [M][K/2]         two 4-bit codes per byte, element 2i in bits 0-3
 *   MXFP4 scales u8 [M][K/32]   E8M0 bytes (e + 127), one per 32 consecutive values
 *   LM4 scales  f32 [M]         per-token scale
 *   mu    fp16 [M]              per-token mean (centring)
 *   W     fp16 [K][N]           weights as in Y = X W (kq_fold_inverse_into_weights);
 *   Wt    fp16 [N][K]           the same weights in the [out][in] layout
 *                               (kq_fold_inverse_into_weights_nk, kq_svd_lowrank)
 *   wcodes u8 [N][K/2] (MXFP4) or [N][K/4] (2-bit, element 4i in bits 0-1)
 *   wscales u8 [N][K/32] (MXFP4) or fp16 [N][K/32] (2-bit group scales)
 *   wbar  fp16 [N]              column sums of W (rank-1 mean restore)
 *   L1    fp16 [r][K], L2 fp16 [N][r]   low-rank factors in the [out][in] layout
 *                               (X L1^T is the down-projection, T L2^T the up-projection:
 *                               the transposes of an L1 [K][r], L2 [r][N] written as
 *                               X L1 L2; rows are contiguous along the contracted
 *                               dimension, which is how the matrix cores take them)
 *   Y     fp16 [M][N]
 *
 * Ownership: the caller allocates and owns every buffer; the library never
 * allocates, frees or caches device memory, and holds no per-call state (it is
 * re-entrant).  Descriptor contents (kind, K, A, B) travel by value; perm, sign, P,
 * AB and pts are caller-owned device arrays.  Every call is asynchronous on `stream` (0 = the
 * null stream); inputs must stay alive until the stream has passed the call.
 *
 * Errors: the return value is a status.  Arguments are validated on the host
 * before anything is launched; a non-zero status means nothing was enqueued
 * (KQ_ERR_HIP: a launch itself failed, reported by hipGetLastError; in a call that
 * launches several kernels, those before the failing one may have been enqueued).  Faults
 * inside kernels surface at the caller's next synchronisation, as HIP defines.
 */
#ifndef KQ_H
#define KQ_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KQ_ABI_VERSION 8

typedef int32_t kq_status;
enum {
  KQ_OK = 0,
  KQ_ERR_NULL = 1,         /* a required pointer is NULL */
  KQ_ERR_SHAPE = 2,        /* M, N < 1; K % 32 != 0; descriptor K != K; bad rank; mu without wbar */
  KQ_ERR_ALIGN = 3,        /* a device pointer is not 16-byte aligned */
  KQ_ERR_UNSUPPORTED = 4,  /* unknown enum, or a size outside the supported range */
  KQ_ERR_VALUE = 5,        /* a transform factor is singular or not finite */
  KQ_ERR_HIP = 6,          /* a HIP launch failed */
  KQ_ERR_WORKSPACE = 7     /* the workspace is missing or smaller than the call needs */
};

/* transform kinds */
enum { KQ_XFORM_NONE = 0, KQ_XFORM_KRON_4X8 = 1, KQ_XFORM_RPBH_32 = 2, KQ_XFORM_DENSE_32 = 3,
       KQ_XFORM_KRON_4X8_BLOCKS = 4 };
/* formats */
enum { KQ_FMT_MXFP4 = 0, KQ_FMT_LM4_TOKEN = 1, KQ_FMT_LM2_G32 = 2 };

/* One layer's block transform.
 * KRON_4X8 (KroQuant §02): every 32-element block x_b of a token is replaced by
 *   x_b . (A (x) B), i.e. with Xm[i][j] = x_b[8i+j]: Ym = A^T Xm B, y_b[8k+l] = Ym[k][l].
 *   A (4x4) and B (8x8) are row-major floats, one pair shared by all blocks.
 * RPBH_32 (OrbitQuant §03): y = x . Pi . blockdiag(H32) . D / sqrt(32) with
 *   (x.Pi)_j = x[perm[j]] over all K, H32 the Sylvester Hadamard matrix
 *   (H[i][j] = (-1)^popcount(i&j)), D = diag(sign), sign[j] in {-1, +1}.
 *   perm (int32 [K], a permutation of 0..K-1) and sign (int8 [K]) are device arrays,
 *   16- and 4-byte aligned.  perm is not checked on the device: an entry outside
 *   0..K-1 gives unspecified codes for that call (the on-chip gather cannot fault).
 * DENSE_32 (KroQuant §01, the block transform P before its Kronecker factorization):
 *   every 32-element block x_b is replaced by x_b . P, P a dense invertible 32x32 matrix
 *   (P: device float32 [32][32], row-major, 16-byte aligned; one P shared by all blocks).
 *   MXFP4 without centring only; the fold inverts P on the device (a singular P gives
 *   non-finite weights).
 * KRON_4X8_BLOCKS (KroQuant §02 with one factor pair per block index): block b of every
 *   token is replaced by x_b . (A_b (x) B_b), same convention as KRON_4X8, with
 *   AB: device float32 [K/32][80], 16-byte aligned; row b holds A_b (16, row-major) then
 *   B_b (64, row-major).  MXFP4 without centring only.  The factors are not checked: a
 *   non-finite entry gives unspecified codes, and the fold inverts each A_b (x) B_b on the
 *   device (a singular one gives non-finite weights for that block).
 * NONE: identity.
 * pts (optional, any kind but RPBH_32; DMQ explainer, channel-wise power-of-two scaling):
 *   device int8 [K], 16-byte aligned, entries e_k in 0..15.  The activation path first
 *   replaces x_k by fp16(x_k 2^-e_k) (round-to-nearest-even; exact unless the result is
 *   subnormal), then transforms; the fold multiplies weight input channel k by 2^e_k
 *   (exact) before the inverse transform, so the product is unchanged.  MXFP4 without
 *   centring only.  Entries are not checked on the device: one outside 0..15 gives
 *   unspecified codes for that call.  NULL: no scaling. */
typedef struct kq_xform {
  int32_t kind;
  int32_t reserved;          /* must be 0 */
  int64_t K;                 /* must equal the K of the call */
  float A[16];
  float B[64];
  const int32_t* perm;
  const int8_t* sign;
  const float* P;            /* DENSE_32 only */
  const float* AB;           /* KRON_4X8_BLOCKS only */
  const int8_t* pts;         /* NULL or per-channel power-of-two exponents */
} kq_xform;

/* KQ_ABI_VERSION of the built library. */
int32_t kq_abi_version(void);

/* Static, human-readable name of a status code (never NULL). */
const char* kq_status_str(kq_status s);

/* Positive levels (ascending) of the symmetric n-level Lloyd-Max quantizer for a
 * unit Gaussian (OrbitQuant §03: one fixed codebook), as the library computes and
 * uses them; n = 4 or 16.  Host memory, n/2 doubles.  Runs on the host only. */
kq_status kq_lloyd_max_levels(int32_t n, double* levels_out);

/* Measurement helper, outside the activation path: the shader clock as the chip runs it
 * (the matrix-core peak scales with it), e.g. while other work occupies the GPU on another
 * stream.  One 64-thread workgroup on `stream` counts shader-clock cycles over spin_us
 * microseconds of the constant 100 MHz reference counter and writes the cycle count and
 * the reference ticks to out[0] and out[1] (device memory, caller-owned, 8-byte aligned);
 * the clock in MHz is 100 out[0] / out[1].  1 <= spin_us <= 1000000. */
kq_status kq_clock_probe(int32_t spin_us, uint64_t* out, hipStream_t stream);

/* Measurement helper, outside the activation path: the rate the scaled FP4 matrix cores
 * sustain with no memory traffic.  `workgroups` workgroups of four wavefronts on `stream`;
 * each wavefront issues `iters` rounds of sixteen independent v_mfma_scale_f32_32x32x64_f8f6f4
 * (E2M1 x E2M1, scales 2^0) on operands a, b read once from `codes` (device, 2048 bytes,
 * 16-byte aligned, caller-owned: lane l's a is bytes 16 l .. 16 l + 15, its b bytes 1024 + 16 l
 * .. ; product u of a round is (u & 1 ? a : b) x (u & 2 ? a : b)) and writes one sum of its
 * accumulators to out[4 * workgroup + wavefront] (device, 4 * workgroups floats,
 * caller-owned).  The work is 64 * iters * workgroups products of 2 * 32 * 32 * 64 flops; the
 * caller times the launch.  1 <= iters <= 1000000, 1 <= workgroups <= 65536. */
kq_status kq_mfma_fp4_probe(int32_t iters, int32_t workgroups, const void* codes, float* out, hipStream_t stream);

/* Online activation path (KroQuant §01-§03; OrbitQuant §03; CentriQ abstract):
 *   [centre]  mu_t = fp16(mean_k X[t,k]) (float32 sum), x <- x - mu_t      if center
 *   transform y = x . P  (xf->kind)
 *   quantize  fmt MXFP4: per 32-block a = max|y|, e = max(floor(log2 a) - 2, -127),
 *                        scale byte e + 127, code = E2M1 round-to-nearest-even of
 *                        y 2^-e, saturating at 6, sign bit = (y < 0); packed.
 *             fmt LM4_TOKEN: s_t = sqrt(mean_k y^2) (float32), code = sign-magnitude
 *                        index of y / s_t in the 16-level Lloyd-Max codebook
 *                        (a value on a threshold takes the smaller magnitude).
 * X fp16 [M][K]; codes u8 [M][K/2]; scales u8 [M][K/32] (MXFP4) or f32 [M] (LM4);
 * mu fp16 [M], required iff center != 0 (else ignored).
 * K % 32 == 0; K <= 16384 when centring, RPBH or LM4 is used (rows are staged on
 * chip).
 * All device pointers 16-byte aligned except mu and scales (4-byte for LM4). */
kq_status kq_transform_quantize(const kq_xform* xf, int32_t fmt, int32_t center,
                                const void* X, int64_t M, int64_t K,
                                uint8_t* codes, void* scales, void* mu,
                                hipStream_t stream);

/* Offline fold (KroQuant §01; OrbitQuant §03 W' = R^-1 W; CentriQ abstract):
 *   W' = P^-1 W (KRON: blockdiag(A^-1 (x) B^-1), the inverses computed on the host in
 *   double precision; RPBH: R^T; DENSE_32 / KRON_4X8_BLOCKS: inverted on the device),
 *   computed in float32 on the device, then each column n of W' (the weights of
 *   output n) quantized along K: fmt MXFP4 with the activation rule, or LM2_G32:
 *   s_g = fp16(RMS of the 32-group), 2-bit sign-magnitude code of w / s_g in the
 *   4-level Lloyd-Max codebook.  wbar[n] = fp16(sum_k W[k][n]) (float64 sum) if
 *   wbar != NULL: the column sums for the rank-1 mean restore.
 * W fp16 [K][N] (row-major: W[k][n] at k*N + n); wcodes u8 [N][K/2] (MXFP4) or [N][K/4]
 * (LM2); wscales u8 [N][K/32] (MXFP4) or fp16 [N][K/32] (LM2); wbar fp16 [N].
 * Untimed: runs once per layer.  Returns KQ_ERR_VALUE if A or B is singular. */
kq_status kq_fold_inverse_into_weights(const kq_xform* xf, int32_t fmt,
                                       const void* W, int64_t K, int64_t N,
                                       uint8_t* wcodes, void* wscales, void* wbar,
                                       hipStream_t stream);

/* The same fold for weights given as Wt fp16 [N][K] (the [out][in] layout, Wt[n][k] =
 * W[k][n]); outputs identical to kq_fold_inverse_into_weights on the same weights. */
kq_status kq_fold_inverse_into_weights_nk(const kq_xform* xf, int32_t fmt,
                                          const void* Wt, int64_t N, int64_t K,
                                          uint8_t* wcodes, void* wscales, void* wbar,
                                          hipStream_t stream);

/* Low-rank down-projection of the 16-bit branch (SVDQuant explainer §3):
 *   T = fp16(X L1^T), fp32 accumulation on the fp16 matrix cores.
 * X fp16 [M][K] (the original activations: not centred, not transformed), L1 fp16 [r][K],
 * T fp16 [M][r] (caller-owned).  r in {16, 32, 48, 64}; K % 32 == 0, K <= 2^20.
 * workspace (optional, caller-owned device memory, 16-byte aligned): when M is small
 *   against the device, K is split over several workgroups whose fp32 partials go to the
 *   workspace, and a second kernel sums them in a fixed order (results do not depend on
 *   scheduling).  kq_lowrank_down_workspace_bytes gives the size that enables the full
 *   split; a smaller workspace gives fewer slices, and NULL / 0 runs unsplit (same
 *   results up to fp32 summation order, slower for small M).  The library allocates
 *   nothing.  Calls that share a workspace must not overlap. */
size_t kq_lowrank_down_workspace_bytes(int64_t M, int64_t K, int32_t r);
kq_status kq_lowrank_down(const void* X, const void* L1, int64_t M, int64_t K, int32_t r,
                          void* T, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* The online activation path and the low-rank down-projection in one pass over X
 * (SVDQuant explainer §3: the 16-bit branch and the 4-bit branch read the same input, and
 * running the branch separately costs an extra read of it):
 *   codes, scales[, mu] = MXFP4 of the (optionally centred) block-transformed X, as
 *                   kq_transform_quantize with fmt MXFP4;
 *   T = fp16(X L1^T) from the original X (neither centred nor transformed), as
 *                   kq_lowrank_down.
 * Kinds NONE, KRON_4X8 and DENSE_32 (no centring): one kernel, X read once.  RPBH_32
 * (centring optional; mu fp16 [M], required iff center != 0): the permutation spans the
 * whole row, so the call runs the row-staged transform and then the down-projection
 * (X is read twice; results equal those of the two separate calls).  No pts.
 * Shapes, layouts, alignment and the workspace rule are those of the two calls it
 * replaces; kq_lowrank_down_workspace_bytes(M, K, r) gives the workspace size.  For the
 * one-kernel kinds, codes may differ from kq_transform_quantize's only at rounding ties of
 * the float32 arithmetic, and T from kq_lowrank_down's only by float32 summation order. */
kq_status kq_transform_quantize_lowrank(const kq_xform* xf, int32_t center, const void* X, int64_t M, int64_t K,
                                        uint8_t* codes, void* scales, void* mu, const void* L1, int32_t r, void* T,
                                        void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Offline rank-r extraction of the 16-bit branch (SVDQuant explainer §3: the weight's
 * leading singular directions stay in 16 bits, the residual is quantized to 4 bits):
 *   W (fp16 [N][K], row n = output n) ~ L2 L1 with L2 = U_r S_r^1/2 (fp16 [N][r]),
 *   L1 = S_r^1/2 V_r^T (fp16 [r][K]) from the r leading singular triplets, and
 *   R = fp16(W - L2 L1) (fp16 [N][K]) computed with the fp16 factors, to be folded and
 *   quantized in place of W (kq_fold_inverse_into_weights; its wbar is then 1^T R).
 *   sigma (optional, float [r]): the singular value estimates, descending.
 * The subspace comes from randomized subspace iteration (Halko, Martinsson and Tropp 2011,
 * algorithms 4.4 / 5.1) started from the caller's omega (float32 [K][l], e.g. Gaussian;
 * the library draws no random numbers) with l - r extra columns and `iters` power steps,
 * re-orthonormalized after every product; float32 products, float64 for the l x l parts.
 * Accuracy depends on the gap between sigma_r and sigma_{l+1} and on iters.
 * r in {16, 32, 64}; r < l <= 96, l <= min(N, K); 0 <= iters <= 16; K % 32 == 0.
 * workspace: caller-owned device memory of kq_svd_lowrank_workspace_bytes(N, K, r, l)
 * bytes, 256-byte aligned; other pointers 16-byte aligned (sigma 4).  Runs several kernels
 * on `stream`; calls sharing a workspace must not overlap. */
size_t kq_svd_lowrank_workspace_bytes(int64_t N, int64_t K, int32_t r, int32_t l);
kq_status kq_svd_lowrank(const void* W, int64_t N, int64_t K, int32_t r, const float* omega, int32_t l,
                         int32_t iters, void* L1, void* L2, void* R, float* sigma, void* workspace,
                         size_t workspace_bytes, hipStream_t stream);

/* The 4-bit linear with its full-precision branches (KroQuant §01: Y = (XP)(P^-1 W);
 * SVDQuant explainer §3: plus the 16-bit low-rank branch X L1 L2; CentriQ abstract: plus
 * the rank-1 mean restore):
 *   Y = Xq . Wq^T  +  (X L1^T) L2^T  +  mu wbar^T          (fp32 accumulate, fp16 out)
 * fmt MXFP4: Xq, Wq MXFP4 (xscales u8 [M][K/32], wscales u8 [N][K/32]); products on
 *   the scaled-FP4 matrix cores, each block pair scaled by 2^(ex+ew).  K % 128 == 0.
 * fmt LM2_G32 (W2A4): Xq per-token Lloyd-Max 4-bit (xscales f32 [M]), Wq 2-bit groups
 *   (wcodes u8 [N][K/4], wscales fp16 [N][K/32]); the codebooks are the library's own
 *   (kq_lloyd_max_levels).  K % 32 == 0.  No low-rank or rank-1 branch (r must be 0).
 * Low-rank branch: X fp16 [M][K] (the original activations, neither centred nor
 *   transformed), L1 fp16 [r][K], L2 fp16 [N][r], r in {0, 16, 32, 48, 64} (0: X, L1,
 *   L2 ignored and may be NULL).  The down-projection T = X L1^T runs first on the
 *   stream (as kq_lowrank_down, T held in the workspace), then one GEMM kernel whose
 *   accumulators start from T L2^T, so the branch adds no pass over Y.
 *   T is rounded to fp16 (the up-projection is an fp16 matrix-core product; the
 *   explainer keeps the branch in 16 bits): the branch then carries a relative error
 *   of at most 2^-11 per T entry, far below the 4-bit product's.
 * Rank-1 restore: mu fp16 [M] and wbar fp16 [N], both or neither.
 * workspace: caller-owned device memory, 256-byte aligned, of at least
 *   kq_w4a4_linear_workspace_bytes(M, r) bytes (0 when r == 0; NULL allowed then).  It
 *   holds T and the split-K partial sums of the down-projection.  The library
 *   allocates nothing.  Calls that share a workspace must not overlap.
 * N % 16 == 0; M <= 2^30, N and K <= 2^20.  Y fp16 [M][N].  Pointers 16-byte aligned,
 *   except xscales and wscales (4) and mu (2).
 * Errors: KQ_ERR_WORKSPACE if r > 0 and the workspace is NULL or too small. */
size_t kq_w4a4_linear_workspace_bytes(int64_t M, int32_t r);
kq_status kq_w4a4_linear(int32_t fmt,
                         const uint8_t* xcodes, const void* xscales, int64_t M, int64_t K,
                         const uint8_t* wcodes, const void* wscales, int64_t N,
                         const void* X, const void* L1, const void* L2, int32_t r,
                         const void* mu, const void* wbar,
                         void* Y, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* For callers that cannot allocate (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc): kq_w4a4_linear without a workspace argument.  T and the
 * down-projection's split-K partial sums live in a fixed device array of
 * KQ_NOALLOC_SCRATCH_BYTES inside the library (one per GPU, held until the process ends);
 * the call allocates nothing and calls no allocating routine.  Rejected with
 * KQ_ERR_WORKSPACE when T alone (M * r * 2 bytes, rounded up to 256) exceeds that size;
 * when T fits but the partial sums of the full split do not, fewer K slices are used
 * (results then differ from kq_w4a4_linear's only in float32 summation order).
 * Every call on a GPU shares that GPU's array: calls that overlap on one GPU (other
 * streams, other threads) race and give undefined results.  Arguments otherwise as
 * kq_w4a4_linear. */
#define KQ_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
kq_status kq_w4a4_linear_noalloc(int32_t fmt,
                                 const uint8_t* xcodes, const void* xscales, int64_t M, int64_t K,
                                 const uint8_t* wcodes, const void* wscales, int64_t N,
                                 const void* X, const void* L1, const void* L2, int32_t r,
                                 const void* mu, const void* wbar,
                                 void* Y, hipStream_t stream);

/* The same linear with the down-projection already done: T fp16 [M][r] from
 * kq_lowrank_down or kq_transform_quantize_lowrank (caller-owned), L2 fp16 [N][r],
 * r in {0, 16, 32, 48, 64} (0: T and L2 ignored).  One kernel launch; no workspace.
 * Other arguments and rules as kq_w4a4_linear. */
kq_status kq_w4a4_linear_t(int32_t fmt,
                           const uint8_t* xcodes, const void* xscales, int64_t M, int64_t K,
                           const uint8_t* wcodes, const void* wscales, int64_t N,
                           const void* T, const void* L2, int32_t r,
                           const void* mu, const void* wbar,
                           void* Y, hipStream_t stream);

/* ---- The 8-bit path: for the layers that 4 bits are too few for, and for the norm and the
 * gated feed-forward block around them.  Values are E4M3 (OCP; 1 sign, 4 exponent, 3 mantissa
 * bits, largest 448) with one E8M0 scale for every 128 consecutive values of a row:
 *   codes  u8 [rows][K]                    E4M3
 *   scales u8 [rows][kq_fp8_scale_cols(K)] byte e + 127 of each group, zero bytes behind the
 *                                          last group (a row is 4 ceil(K / 512) bytes)
 * K is a multiple of 16; the last group of a row may be short.  A group's e is the smallest
 * with max|y| <= 448 2^e (at least -127), its codes are y 2^-e rounded to nearest even; a
 * group of zeros has byte 0.  A group that holds an infinity or a NaN has byte 255 and code
 * 0x7F throughout (both NaN), and makes NaN every product that uses it.
 * Codes and scales from elsewhere may be used if every value code 2^e is zero or a normal
 * float32 number (others may over- or underflow to infinity or zero).
 * Weights are [N][K] ([out][in]) and are quantized by the same call as activations; scales
 * given for blocks of 128 x 128 are the special case in which 128 rows repeat the same bytes.
 * 16-bit inputs and outputs are fp16 or bf16 (KQ_DT_*), sums are float32.  M <= 2^30; N and
 * K <= 2^20, F <= 2^19, all multiples of 16.  Pointers 16-byte aligned, scales 4, workspaces
 * 256.  Outputs must not overlap inputs or each other, except where a call says so.  The
 * current device must be the one that the stream and the pointers belong to. */
enum { KQ_DT_F16 = 0, KQ_DT_BF16 = 1 };
enum { KQ_ACT_SILU = 0, KQ_ACT_GELU = 1, KQ_ACT_GELU_TANH = 2 };
/* Or'ed into the dtype of kq_attention: see there.  Or'ed into the dtype of kq_fp8_linear or the act of
 * kq_fp8_gated_linear: every product of two codes exact and added in float32, as calls of up to 16 tokens
 * always do, and a gated call's activation by
 * the library's exponential and a rounded quotient.  Without it, calls of more tokens use the 8-bit matrix
 * instructions, which cut off (towards zero) each of eight consecutive products at 2^(E - 13), E the largest
 * of the eight's sums of two exponents (a subnormal code's exponent is that of the smallest normal one).
 * So a sum is off by at most 7 * 2^(E - 13) added over the eights; relative to the sum itself there is no
 * bound (p, -p and a much smaller q in one eight lose q).  Norm of the errors over norm of the sums, measured:
 * 1.0e-5 to 1.6e-5 on Gaussian values, 2e-5 to 7e-5 with 12 channels of 20 times the size (K = 16 to
 * 11008), 1e-8 to 2e-7 with the flag.  It costs 1 to 10% up to 32 tokens and, for long prompts, as much
 * time again. */
enum { KQ_FP8_PRECISE = 0x100 };

/* Bytes of a row of scales, 4 ceil(K / 512); 0 for a K outside 1 .. 2^20. */
int64_t kq_fp8_scale_cols(int64_t K);

/* codes, scales of X [M][K] (activations with no norm before them, and weights offline). */
kq_status kq_quantize_fp8(int32_t dtype, const void* X, int64_t M, int64_t K, uint8_t* codes, uint8_t* scales,
                          hipStream_t stream);

/* Residual addition, root-mean-square norm and quantization in one pass:
 *   h = X + residual (float32; h = X if residual is NULL),
 *   residual_out = h rounded to the dtype (written only if residual is given),
 *   codes, scales of y = h / sqrt(mean_k h^2 + eps) * gamma.
 * y is formed from the float32 h, not from its rounded copy.  All 16-bit arrays have the one
 * dtype: X, residual, residual_out [M][K], gamma [K].  residual_out may be residual itself.
 * K <= 16384 (a row stays in registers); eps finite and >= 0 (else KQ_ERR_VALUE).  Rows
 * of any finite size are normalized, to float32's ends; a row of zeros with eps = 0 gives NaN. */
kq_status kq_rmsnorm_quantize_fp8(int32_t dtype, const void* X, const void* residual, const void* gamma, float eps,
                                  int64_t M, int64_t K, uint8_t* codes, uint8_t* scales, void* residual_out,
                                  hipStream_t stream);

/* Y = Xq Wq^T (+ bias): Y [M][N] and bias [N] (or NULL) in the dtype, float32 accumulation (of exact
 * products to 16 tokens or with KQ_FP8_PRECISE, which says what the others lose: a tenth of fp16's own
 * rounding).  The order of additions is fixed: equal inputs of equal shape give equal bits. */
kq_status kq_fp8_linear(int32_t dtype, const uint8_t* xcodes, const uint8_t* xscales, int64_t M, int64_t K,
                        const uint8_t* wcodes, const uint8_t* wscales, int64_t N, const void* bias, void* Y,
                        hipStream_t stream);

/* The first half of a gated feed-forward block: codes, scales ([M][F]) of
 *   act(Xq Wg^T) * (Xq Wu^T),   wcodes [2 F][K]: the F rows of Wg, then the F rows of Wu.
 * act: SiLU g / (1 + exp -g); GELU g Phi(g); its tanh form; with or without KQ_FP8_PRECISE.  Both projections, the activation
 * and the product stay in float32; the result is rounded once, to E4M3.  kq_fp8_linear with
 * the down-projection's weights takes codes and scales as they are.  workspace: at least
 * kq_fp8_gated_linear_workspace_bytes(M, F, K) bytes (0: none needed), which holds the float32
 * outputs of a few tokens (up to 32, and up to 64 as far as the device's compute units hold the workgroups:
 * ask on the device that runs the call).  Calls that share a workspace must not overlap, replays of captured
 * graphs that hold it included. */
size_t kq_fp8_gated_linear_workspace_bytes(int64_t M, int64_t F, int64_t K);
kq_status kq_fp8_gated_linear(int32_t act, const uint8_t* xcodes, const uint8_t* xscales, int64_t M, int64_t K,
                              const uint8_t* wcodes, const uint8_t* wscales, int64_t F, uint8_t* codes,
                              uint8_t* scales, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ---- Attention of the 8-bit path: between the projection of queries, keys and values and the output
 * projection.  16-bit types are fp16 or bf16 (KQ_DT_*), one in all 16-bit arrays of a call.  Hq query heads
 * share Hkv key heads, Hq / Hkv at a time (head h reads key head h Hkv / Hq); D values a head, a multiple of
 * 8, 8 to 128.
 *
 *   o = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q . k_j - max),  over the keys j that the query sees;
 *
 * a query that sees no key (or none with a score above minus infinity) gets zeros, and what is at keys that
 * it does not see (NaN and infinities included) does not reach it.  Scores, maxima and sums are float32.  For the
 * product with the values kq_attention rounds a weight to the 16-bit type (relative error 2^-8 bf16, 2^-11 fp16), which
 * moves 16-bit outputs by less than their own rounding, and codes by 0.2 to 1% of the norm (E4M3 itself 2.7%).
 * kq_paged_attention, and kq_attention with KQ_FP8_PRECISE or'ed into its dtype, multiply it as a sum of 16-bit
 * numbers: two of fp16 (2^-22) for fp16 keys and values, else three of bf16 (2^-24); codes are then as near 64 bits as
 * with float32 throughout (0.02% of the norm).  Prompts take 1.1 to 1.9 times as long so.  What a weight loses besides is below 2^-31 of the largest (fp16) or 2^-125; one that
 * vanishes makes NaN of an infinite value.  Sums are divided by the weights' sum at the end, so values beyond 10^30
 * may overflow.  The order of additions is fixed for one device: equal inputs of equal shape give equal bits.
 *
 * Outputs: O [rows][Hq][D] in the 16-bit type, or, where codes and scales are given instead (O NULL; D = 128
 * only), E4M3 codes [rows][Hq 128] with one E8M0 byte for each head, [rows][kq_fp8_scale_cols(Hq 128)],
 * rounded once from float32: what kq_fp8_linear takes.  Contiguous.  Pointers 16-byte aligned, integers,
 * table and scales 4.  Entries of device arrays (cu, table, lengths) are not checked on the host; kernels hold
 * them to what the arrays can hold, as each call says, so none leads out of them. */

/* Packed sequences: sequence s has queries cu_q[s] .. cu_q[s + 1] - 1 of Q and keys cu_k[s] .. cu_k[s + 1] - 1 of
 * K and V (cu_q, cu_k: int32 [B + 1], ascending, device memory; both NULL: one sequence of T queries and Tk keys,
 * B = 1).  causal: query i of a sequence sees the keys j <= i + Lk - Lq, so the last query sees all.  Rows of Q
 * outside all sequences get no output: theirs is left as it was.  Entries of cu are held to 0 .. T (Tk)
 * and to their order.
 * Q, K, V: element (token, head, d) at token * token stride + head * head stride + d, strides in elements,
 * multiples of 8; token strides D to 2^21, head strides 0 to 2^40.  Views of one projection's output
 * [T][(Hq + 2 Hkv) D] are the usual case.  1 <= T, Tk <= 2^30 (a sequence may have no
 * queries or no keys; a call may not), T Hq <= 2^29, 1 <= B, B Hq <= 2^22.  scale finite, above 0.
 * workspace: at least kq_attention_workspace_bytes bytes (packed: whether cu is given), 256-byte aligned (0: none needed, as
 * for Tk <= 704 whatever else; few queries of more keys are split over the keys, and it holds the parts.  It depends on the device's compute units:
 * ask on the device that runs the call).  Calls that share a workspace must not overlap, replays of captured
 * graphs that hold it included. */
size_t kq_attention_workspace_bytes(int64_t B, int64_t T, int64_t Tk, int32_t packed, int32_t Hq, int32_t Hkv, int32_t D);
kq_status kq_attention(int32_t dtype, const void* Q, int64_t q_token, int64_t q_head, const void* K, int64_t k_token,
                       int64_t k_head, const void* V, int64_t v_token, int64_t v_head, const int32_t* cu_q,
                       const int32_t* cu_k, int64_t B, int64_t T, int64_t Tk, int32_t Hq, int32_t Hkv, int32_t D,
                       int32_t causal, float scale, void* O, uint8_t* codes, uint8_t* scales, void* workspace,
                       size_t workspace_bytes, hipStream_t stream);

/* A cache of keys and values in pages of `page` tokens (a multiple of 16, to 65536): kcache, vcache
 * [pages][Hkv][page][D], in the 16-bit type; or, with kscales and vscales (both or neither; [pages][Hkv][page]),
 * E4M3 codes with one E8M0 byte for each token and head, as kq_quantize_fp8 would give for a row of D
 * values (D a multiple of 16 then).  table int32 [B][width] names each sequence's pages in order, lengths
 * int32 [B] its tokens; lengths are held to 0 .. width * page, and entries of the table outside 0 .. pages - 1
 * are pages that are not there: their tokens are neither written nor seen.  Entries behind a sequence's last
 * page are not read.  A page may be in several sequences' tables (a common beginning); one that receives
 * tokens must be in one.  B <= 2^20, width * page <= 2^30, B width page <= 2^37, pages < 2^31. */

/* Writes new tokens' keys and values: lengths already count them.  Sequence s's new tokens are rows cu[s] ..
 * cu[s + 1] - 1 of K and V (int32 [B + 1], ascending; NULL: one token each, T = B), the last of them at
 * position lengths[s] - 1.  K, V: as kq_attention, head strides to 2^40.  Tokens whose position is
 * outside the table, and rows outside all sequences, are not written.  1 <= T <= 2^25. */
kq_status kq_cache_append(int32_t dtype, const void* K, int64_t k_token, int64_t k_head, const void* V, int64_t v_token,
                          int64_t v_head, const int32_t* cu, int64_t B, int64_t T, int32_t Hkv, int32_t D,
                          const int32_t* table, int64_t width, const int32_t* lengths, void* kcache, void* vcache,
                          uint8_t* kscales, uint8_t* vscales, int64_t pages, int32_t page, hipStream_t stream);

/* One new token a sequence: query b of Q [B][Hq][D] (strides as above, both D to 2^21) sees the lengths[b]
 * tokens of its sequence.  workspace: at least kq_paged_attention_workspace_bytes bytes, 256-byte aligned (0: none
 * needed; it depends on the device's compute units: ask on the device that runs the call).  Calls that share a workspace
 * must not overlap, replays of captured graphs that hold it included.  B Hq <= 2^23.  scale finite, above 0. */
size_t kq_paged_attention_workspace_bytes(int64_t B, int32_t Hq, int32_t Hkv, int32_t D, int64_t width, int32_t page);
kq_status kq_paged_attention(int32_t dtype, const void* Q, int64_t q_seq, int64_t q_head, const void* kcache,
                             const void* vcache, const uint8_t* kscales, const uint8_t* vscales, int64_t pages,
                             int32_t page, const int32_t* table, int64_t width, const int32_t* lengths, int64_t B,
                             int32_t Hq, int32_t Hkv, int32_t D, float scale, void* O, uint8_t* codes, uint8_t* scales,
                             void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* KQ_H */
