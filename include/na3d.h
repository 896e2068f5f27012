/*
 * na3d.h - C ABI of the GB300 (sm_103a) forward pass of 3-D neighborhood
 * attention (NA3D).
 *
 * The operation ("[Triton/Gluon] Add 3D neighborhood flash attention
 * (na3d_flash)", ROCm/aiter pull request 5230):
 *   - Motivation: the token at grid position (t,h,w) of a video latent
 *     attends only to its KT x KH x KW neighbours.
 *   - Technical Details, kernel bullets: windows shift inward at the grid
 *     borders so that every window holds exactly KT*KH*KW keys; the softmax
 *     runs online in log2 space.
 *   - Technical Details, launcher: inputs and output are (B, T, H, W, NH, HD)
 *     bfloat16, and q arrives already multiplied by head_dim^-0.5.
 *
 * On each axis of length N with odd window length K <= N, the query at i uses
 * keys [s, s+K) with s = min(max(i - K/2, 0), N - K) (integer division).
 * Scores are q.k accumulated in fp32, the softmax over the window runs in
 * fp32, the probabilities are rounded to bf16 for the P.V product (fp32
 * accumulation), and the output is rounded to bf16 (nearest even).
 *
 * The library allocates no memory and is safe to call from several host
 * threads at once. Its only state is two caches of tiling plans (keyed by grid
 * and window sizes; one guarded by a mutex, the na3d_scored_ calls' one kept by
 * each thread) and, per device and kernel family, one word that records a
 * pipeline-wait timeout plus the small table of words through which
 * na3d_device_status takes it (see there).
 */
#ifndef NA3D_H
#define NA3D_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes returned by every entry point. */
enum na3d_status {
    NA3D_OK = 0,
    NA3D_ERR_NULL = 1,           /* a required pointer is NULL */
    NA3D_ERR_SHAPE = 2,          /* a size < 1, or a query box outside the grid */
    NA3D_ERR_KERNEL = 3,         /* a window length is even, < 1, or larger than its axis */
    NA3D_ERR_HEAD_DIM = 4,       /* HD is not a power of two >= 16 */
    NA3D_ERR_ALIGN = 5,          /* a tensor pointer is not 16-byte aligned */
    NA3D_ERR_ALIAS = 6,          /* out overlaps q, k or v */
    NA3D_ERR_OVERFLOW = 7,       /* a size overflows int64 or a TMA descriptor limit */
    NA3D_ERR_ARCH = 8,           /* the current device is not compute capability 10.3 */
    NA3D_ERR_CUDA = 9,           /* a CUDA runtime or driver call failed */
    NA3D_ERR_DEVICE_TIMEOUT = 10, /* a pipeline wait inside the kernel gave up */
    NA3D_ERR_UNSUPPORTED = 11    /* valid but not implemented: HD > 128 or a softcap outside its range in
                                     the na3d_scored_ calls, R > 128 in the na3d_lora_ calls */
};

/*
 * na3d_fwd - out = NA3D(q, k, v) for one bf16 (B,T,H,W,NH,HD) problem.
 *
 * The operation of "[Triton/Gluon] Add 3D neighborhood flash attention
 * (na3d_flash)" (ROCm/aiter pull request 5230), Technical Details: the query
 * at (t,h,w) attends to the KT x KH x KW keys of its window, shifted inward at
 * the grid borders so that it always holds KT*KH*KW keys (the start rule is
 * stated at the top of this file); the launcher's convention that q arrives
 * already multiplied by head_dim^-0.5 and that inputs and output share the
 * (B,T,H,W,NH,HD) bf16 layout.
 *
 * q, k, v, out: DEVICE pointers to contiguous row-major bf16 tensors of shape
 *   (B, T, H, W, NH, HD) (HD fastest), each 16-byte aligned. The caller owns
 *   all four buffers; the library neither allocates nor frees memory.
 *   q must already be scaled by HD^-0.5: no scale is applied. q, k and v are
 *   read only and may alias one another; out must not overlap any of them.
 * B: batch size, T, H, W: grid sizes, NH: heads, all >= 1 (a size < 1,
 *   including an empty batch, returns NA3D_ERR_SHAPE).
 * HD: head dimension, a power of two >= 16, with NH*HD < 2^31 (else
 *   NA3D_ERR_OVERFLOW). Above 256 the output is computed in passes of 256
 *   columns that recompute the same scores (slower per column, same result).
 * KT, KH, KW: odd window lengths with 1 <= KT <= T, 1 <= KH <= H, 1 <= KW <= W.
 * stream: a cudaStream_t on the current device (NULL = legacy default stream).
 *
 * The call validates its arguments, encodes the TMA descriptors on the host
 * and enqueues one kernel on `stream`; it returns before the kernel runs. An
 * argument error returns its code before anything is enqueued (out is not
 * written). NA3D_ERR_CUDA reports a failed launch or descriptor encoding.
 * Faults inside the kernel surface through the stream as usual; a pipeline
 * wait that gives up is reported by na3d_device_status(). The launch may be
 * captured into a CUDA graph on `stream` (the tensor maps are passed by
 * value and the plan is chosen at capture time); replays read the buffers
 * the call was given. na3d_device_status synchronizes and cannot be captured.
 */
int na3d_fwd(const void* q, const void* k, const void* v, void* out,
             int64_t B, int64_t T, int64_t H, int64_t W, int64_t NH, int64_t HD,
             int64_t KT, int64_t KH, int64_t KW, void* stream);

/*
 * na3d_fwd_strided - na3d_fwd for inputs whose grid positions are not packed:
 * q, k and v each hold, for token p = ((b*T + t)*H + h)*W + w, its NH heads
 * of HD values at  base + p*token_stride + head*HD  (elements). This is the
 * layout of a fused QKV projection output [B,T,H,W,3,NH,HD]: token_stride =
 * 3*NH*HD, with q, k, v pointing at the three blocks of the first token, so
 * the projection output feeds the attention without a gather copy (the
 * copy the pages' benchmark pays: "[Triton/Gluon] Add 3D neighborhood flash
 * attention (na3d_flash)", Performance table, "times include the wrapper's
 * v.contiguous() staging copy").
 *
 * q_token_stride, k_token_stride, v_token_stride: >= NH*HD, in elements; a
 * stride times 2 bytes must be a multiple of 16. out stays contiguous
 * (B,T,H,W,NH,HD) and must not overlap the memory spanned by q, k or v.
 * All other arguments, the errors and the asynchrony are those of na3d_fwd;
 * a bad stride returns NA3D_ERR_SHAPE (too small) or NA3D_ERR_ALIGN.
 */
int na3d_fwd_strided(const void* q, const void* k, const void* v, void* out,
                     int64_t B, int64_t T, int64_t H, int64_t W, int64_t NH, int64_t HD,
                     int64_t KT, int64_t KH, int64_t KW, int64_t q_token_stride,
                     int64_t k_token_stride, int64_t v_token_stride, void* stream);

/*
 * na3d_fwd_region - queries on a box of the grid, keys and values on the whole
 * grid: out = NA3D(q, k, v) restricted to the grid positions (t0 + t, h0 + h,
 * w0 + w), 0 <= t < Tq, 0 <= h < Hq, 0 <= w < Wq. Every query keeps the window
 * it has in the whole grid (global coordinates, shifted inward at the grid's
 * borders, never at the box's), so the result equals the matching rows of
 * na3d_fwd on the whole grid. This generalises the test reference's
 * `w_offset` mode ("[Triton/Gluon] Add 3D neighborhood flash attention
 * (na3d_flash)", Technical Details, test file: q a W sub-slice, k and v the
 * full tensors, bounds in global W coordinates) to a box on all three axes:
 * tiles of a decoded video are computed with exact borders.
 *
 * q: (B, Tq, Hq, Wq, NH, HD) tokens with q_token_stride elements between
 *   consecutive positions of the box (heads packed).
 * k, v: (B, T, H, W, NH, HD), the whole grid, with k_token_stride and
 *   v_token_stride elements between consecutive grid positions.
 * out: contiguous (B, Tq, Hq, Wq, NH, HD); must not overlap the memory that
 *   q, k or v span.
 * t0, h0, w0 >= 0 and Tq, Hq, Wq >= 1 with t0 + Tq <= T, h0 + Hq <= H,
 *   w0 + Wq <= W; otherwise NA3D_ERR_SHAPE. Windows satisfy KT <= T,
 *   KH <= H, KW <= W (the box may be narrower than a window).
 * All other arguments, the errors and the asynchrony are those of
 * na3d_fwd_strided; na3d_fwd_strided is this call with the whole grid as the
 * box (t0 = h0 = w0 = 0, Tq = T, Hq = H, Wq = W).
 */
int na3d_fwd_region(const void* q, const void* k, const void* v, void* out,
                    int64_t B, int64_t T, int64_t H, int64_t W, int64_t NH, int64_t HD,
                    int64_t KT, int64_t KH, int64_t KW,
                    int64_t t0, int64_t h0, int64_t w0, int64_t Tq, int64_t Hq, int64_t Wq,
                    int64_t q_token_stride, int64_t k_token_stride, int64_t v_token_stride,
                    void* stream);

/*
 * na3d_qkv_proj - the fused QKV projection that feeds the attention:
 *   qkv[m][n] = bf16( s_n * ( sum_c x[m][c] * w[n][c] + bias[n] ) ),
 *   s_n = HD^-0.5 (rounded to fp32) for n < NH*HD (the q block), else 1,
 * with the sum and the bias added in fp32 and one rounding to bf16 (nearest
 * even). The decoder attention of "LTX-2.5 optimization: integrate faster
 * AITER NA3D flash attention for diffusion decoder" (xDiT pull request 773,
 * Summary; Notes) projects q, k and v with one concatenated weight and takes
 * q, k, v as views of the result; the attention wants q already scaled by
 * HD^-0.5 ("[Triton/Gluon] Add 3D neighborhood flash attention (na3d_flash)",
 * Technical Details, launcher). A row of qkv is [q heads | k heads | v heads],
 * i.e. (M, 3, NH, HD): pass qkv, qkv + NH*HD and qkv + 2*NH*HD (elements) to
 * na3d_fwd_strided with token strides 3*NH*HD, and M = B*T*H*W tokens in
 * (b, t, h, w) order.
 *
 * x: DEVICE pointer, bf16 (M, C) row-major (a token's C input channels).
 * w: DEVICE pointer, bf16 (3*NH*HD, C) row-major (one output feature per
 *   row, as a linear layer's weight), q rows first, then k, then v.
 * bias: DEVICE pointer, bf16 (3*NH*HD), or NULL for none.
 * qkv: DEVICE pointer, bf16 (M, 3*NH*HD) row-major; must not overlap x, w or
 *   bias. x, w and qkv are 16-byte aligned; C is a multiple of 8 (16-byte
 *   rows), else NA3D_ERR_ALIGN.
 * M >= 1 tokens, NH >= 1 heads, C >= 1 (else NA3D_ERR_SHAPE), HD a power
 *   of two >= 16.
 * Asynchronous on `stream`; errors as for na3d_fwd. na3d_device_status also
 * reports a pipeline wait of this kernel that gave up.
 */
int na3d_qkv_proj(const void* x, const void* w, const void* bias, void* qkv,
                  int64_t M, int64_t C, int64_t NH, int64_t HD, void* stream);

/*
 * na3d_scored_fwd - neighborhood attention whose scores are shaped before the
 * softmax, on a batch that may pack several clips into one grid. Query i sees
 * the keys j of its window (the window of na3d_fwd, on the whole grid); with
 * a = q_i . k_j,
 *   s = a, or softcap * tanh(a / softcap) where softcap > 0,
 *   s -= slopes[head][0] |t_i - t_j| + slopes[head][1] |h_i - h_j|
 *        + slopes[head][2] |w_i - w_j|                 (slopes not NULL),
 * and key j is masked
 *   - where doc_i != doc_j or doc_i < 0                (doc not NULL): clips
 *     do not see one another, and a position with a negative document is
 *     padding, which sees nothing and is seen by nothing;
 *   - where t_j > t_i and t_j >= prefix[b]             (prefix not NULL):
 *     causal along T, with the first prefix[b] frames seen by every frame.
 * The masks cut a window that is taken on the whole grid. So a clip that is
 * packed with others, or padded, is not the clip by itself within half a
 * window of the cut: alone its windows would shift inward and hold all their
 * KT * KH * KW keys, here they hold those on the clip's side. Farther from a
 * cut the rows are equal. prefix counts from the entry's first frame: of the
 * clips packed along T into one entry only the first can have one.
 * out_i = sum_j p_ij v_j with p the softmax of the s that are not masked, and
 * lse_i = log sum_j e^s. A row that sees nothing has out 0 and lse -infinity.
 * What masked keys and padding hold (infinities and NaN included) reaches no
 * row that does not see them; values that are not finite cost time, though,
 * since the rows about them are computed one by one. Sums, statistics and
 * probabilities are fp32; the probabilities are rounded to bf16 for their
 * product with v, out is rounded once. Under a cap a score, and with it lse, is
 * off by up to 2^-21 of the cap beside 2^-19 of the magnitudes in its sums.
 *
 * q (scaled by HD^-0.5), k, v: bf16 with a token stride, as
 *   na3d_fwd_strided; out: contiguous (B,T,H,W,NH,HD).
 * lse: fp32 (B,T,H,W,NH), or NULL; the backward pass needs it.
 * softcap: 0 (none) or 2^-10 .. 2^20, else NA3D_ERR_UNSUPPORTED.
 * slopes: fp32 (NH, 3) or NULL; doc: int32 (B,T,H,W) or NULL; prefix: int32
 *   (B) or NULL. All DEVICE pointers, 4-byte aligned, read when the kernels
 *   run (a replayed graph sees their current contents).
 * HD: 16, 32, 64 or 128; other powers of two return NA3D_ERR_UNSUPPORTED.
 * Windows: the masks of a frame's part of a window lie in shared memory. Up to
 *   KH * KW = 2^14 keys they always fit; larger windows that do not (from about
 *   28000 keys on, by shape and pass) return NA3D_ERR_UNSUPPORTED, and so do
 *   grids of more than 2^31 - 1 tiles of up to 16 rows and KT above 2^23.
 * out and lse must not overlap an input or one another. All other arguments,
 * the errors, the asynchrony and the capture into graphs are those of
 * na3d_fwd_strided.
 */
int na3d_scored_fwd(const void* q, const void* k, const void* v, void* out, float* lse,
                    int64_t B, int64_t T, int64_t H, int64_t W, int64_t NH, int64_t HD,
                    int64_t KT, int64_t KH, int64_t KW, int64_t q_token_stride,
                    int64_t k_token_stride, int64_t v_token_stride, float softcap,
                    const float* slopes, const int32_t* doc, const int32_t* prefix,
                    void* stream);

/*
 * na3d_scored_bwd - the gradients of na3d_scored_fwd. With p = e^(s - lse),
 * dp = dout_i . v_j, delta_i = dout_i . out_i and
 * da = p (dp - delta_i) (1 - tanh(a / softcap)^2)   (the last factor 1 without a cap),
 *   dq_i = sum_j da k_j,   dk_j = sum_i da q_i,   dv_j = sum_i p dout_i.
 * dq is the gradient of the scaled q that was passed. slopes, doc and prefix
 * are constants. The sums have a fixed order: equal inputs give equal bits.
 * p and da are rounded to bf16 for their products (fp32 sums; for dq da is
 * kept in two such parts), the gradients once at the end. The delta of dq has
 * the rounding of out in it, but for windows of up to five keys.
 *
 * out, lse: what na3d_scored_fwd wrote for the same arguments; dout: bf16,
 *   contiguous (B,T,H,W,NH,HD).
 * dq, dk, dv: bf16 with token strides (the three blocks of a fused
 *   (B,T,H,W,3,NH,HD) gradient, for instance); written whole, padding's
 *   gradients as 0. They must not share elements with one another or overlap
 *   an input or the workspace.
 * work: DEVICE workspace of na3d_scored_bwd_workspace() bytes, 16-byte
 *   aligned, its contents arbitrary; in use until the call's kernels end, so
 *   calls that may run at the same time need their own.
 * All other arguments and errors are those of na3d_scored_fwd.
 */
int na3d_scored_bwd(const void* q, const void* k, const void* v, const void* out,
                    const float* lse, const void* dout, void* dq, void* dk, void* dv, void* work,
                    int64_t B, int64_t T, int64_t H, int64_t W, int64_t NH, int64_t HD,
                    int64_t KT, int64_t KH, int64_t KW, int64_t q_token_stride,
                    int64_t k_token_stride, int64_t v_token_stride, int64_t dq_token_stride,
                    int64_t dk_token_stride, int64_t dv_token_stride, float softcap,
                    const float* slopes, const int32_t* doc, const int32_t* prefix,
                    void* stream);

/* Bytes of workspace of na3d_scored_bwd; -1 where a size is invalid. */
int64_t na3d_scored_bwd_workspace(int64_t B, int64_t T, int64_t H, int64_t W, int64_t NH);

/*
 * na3d_lora_qkv_proj - na3d_qkv_proj with a low-rank adapter for each request
 * of the batch. Rows offsets[r] <= m < offsets[r+1] belong to request r, whose
 * adapter is a = adapter[r]:
 *   t[m] = scaling[a] * ( x[m] A_a^T )                      (R values)
 *   qkv[m][n] = bf16( s_n * ( sum_c x[m][c] w[n][c] + bias[n] + sum_r t[m][r] B_a[n][r] ) )
 * with s_n as in na3d_qkv_proj. Rows outside every request, and requests whose
 * id is not in 0 .. n_adapters - 1 (-1, say), get the base projection alone;
 * several requests may name one adapter. All sums are fp32; t is rounded to
 * bf16 for its product with B_a.
 *
 * x, w, bias, qkv, M, C, NH, HD: as na3d_qkv_proj.
 * lora_a: DEVICE, bf16 (n_adapters, R, C); lora_b: DEVICE, bf16
 *   (n_adapters, 3*NH*HD, R), 16-byte aligned. An adapter of lower rank is
 *   padded with zeros. R: a multiple of 8 (else NA3D_ERR_ALIGN) up to 128 (else
 *   NA3D_ERR_UNSUPPORTED).
 * scaling: DEVICE, fp32 (n_adapters).
 * offsets: DEVICE, int32 (n_requests + 1), not decreasing, within 0 .. M;
 *   adapter: DEVICE, int32 (n_requests). Both are read when the kernels run,
 *   so a replayed graph may be given other requests. Offsets that decrease or
 *   leave 0 .. M touch no memory outside the tensors, but the values are then
 *   unspecified.
 * n_requests, n_adapters >= 1; n_requests up to M + 2^20, else
 *   NA3D_ERR_UNSUPPORTED (more are empty, and a tile's are walked one by one).
 * work: DEVICE workspace of na3d_lora_workspace(..., 0) bytes, 16-byte aligned,
 *   contents arbitrary; as in na3d_scored_bwd, one call at a time.
 * qkv and work must not overlap an input or one another. Errors, asynchrony
 * and capture as na3d_qkv_proj.
 */
int na3d_lora_qkv_proj(const void* x, const void* w, const void* bias, const void* lora_a,
                       const void* lora_b, const float* scaling, const int32_t* offsets,
                       const int32_t* adapter, void* qkv, void* work, int64_t M, int64_t C,
                       int64_t NH, int64_t HD, int64_t R, int64_t n_requests,
                       int64_t n_adapters, void* stream);

/*
 * na3d_lora_qkv_proj_bwd - the gradients of na3d_lora_qkv_proj with a frozen
 * base weight, bias and scaling. With g = s_n dqkv and, for each row's
 * adapter, u = scaling[a] * ( g B_a ):
 *   dx = g W + u A_a,
 *   dlora_a[a] = sum over the adapter's rows of u^T x,
 *   dlora_b[a] = sum over the adapter's rows of g^T t.
 * Sums are fp32 in a fixed order; t and u are rounded to bf16 for their
 * products, the results once at the end. An adapter that no row has gets
 * zeros.
 *
 * dqkv: DEVICE, bf16 (M, 3*NH*HD), 16-byte aligned.
 * dx: bf16 (M, C), or NULL where it is not wanted; dlora_a, dlora_b: as lora_a,
 *   lora_b; all written whole, 16-byte aligned.
 * work: na3d_lora_workspace(..., 1) bytes. No output may overlap an input, the
 * workspace or another output. All other arguments and errors are those of
 * na3d_lora_qkv_proj.
 */
int na3d_lora_qkv_proj_bwd(const void* dqkv, const void* x, const void* w, const void* lora_a,
                           const void* lora_b, const float* scaling, const int32_t* offsets,
                           const int32_t* adapter, void* dx, void* dlora_a, void* dlora_b,
                           void* work, int64_t M, int64_t C, int64_t NH, int64_t HD, int64_t R,
                           int64_t n_requests, int64_t n_adapters, void* stream);

/* Bytes of workspace of na3d_lora_qkv_proj (backward 0) or its backward pass
 * (backward 1); -1 where a size is invalid or not supported. */
int64_t na3d_lora_workspace(int64_t M, int64_t C, int64_t NH, int64_t HD, int64_t R,
                            int64_t n_requests, int64_t n_adapters, int backward);

/*
 * na3d_selftest_withhold - a self-test of the kernel's failure detection:
 * na3d_fwd on contiguous tensors, except that CTA 0 does not issue the load
 * of its K chunk number `chunk` (0-based, in its own order). The score-tile
 * wait for that chunk runs out after about 2 s; the CTA then records the
 * timeout, drains its in-flight copies and MMAs, frees its tensor memory and
 * exits, and na3d_device_status() returns NA3D_ERR_DEVICE_TIMEOUT. out is
 * left partly unwritten. The stream and the device stay usable. Not for
 * production use. chunk < 0 returns NA3D_ERR_SHAPE; other arguments and
 * errors as na3d_fwd.
 */
int na3d_selftest_withhold(const void* q, const void* k, const void* v, void* out,
                           int64_t B, int64_t T, int64_t H, int64_t W, int64_t NH, int64_t HD,
                           int64_t KT, int64_t KH, int64_t KW, int64_t chunk, void* stream);

/* Human-readable name of a status code (static storage, never NULL). */
const char* na3d_status_string(int status);

/*
 * How na3d_fwd tiles one (batch, head) slice: queries are cut into bricks of
 * bt x bh x bw grid positions (at most 128 queries, one tile of the tensor
 * cores), and each brick streams the union of its queries' windows (its halo)
 * through shared memory in chunks of cr rows (consecutive h) of cw keys
 * (consecutive w) in one frame t. The scores of a chunk form one
 * 128 x n_mma tile (n_mma <= tile_cap).
 */
typedef struct na3d_plan_info {
    int32_t bt, bh, bw;           /* query brick */
    int32_t cw, cr;               /* chunk: cr rows of cw keys */
    int32_t n_mma;                /* score-tile width (cr*cw rounded up to 16) */
    int32_t hd_box;               /* head-dim columns per TMA box (HD or 64) */
    int32_t stages;               /* K/V shared-memory pipeline depth */
    int64_t bricks_per_slice;     /* bricks per (batch, head) slice */
    int64_t chunks_per_slice;     /* chunks per (batch, head) slice */
    int64_t smem_bytes;           /* dynamic shared memory per CTA */
    int32_t w_stride;             /* 8, 12, 14, 16 or 32: chunk rows padded to this many keys
                                     and the W window applied by the tensor core (12 and 14
                                     for HD 64 and 128 only); 1: every W window
                                     is the whole axis (KW == W), chunk rows are whole grid
                                     rows and the H window is applied by the tensor core;
                                     0: per-key masks */
    int32_t tile_cap;             /* score-tile capacity of the kernel instance: 128 (HD <= 64) or
                                     64 (HD >= 128), or 96 for the HD <= 64 instances whose score
                                     tiles are double-buffered (the next one is computed while
                                     the softmax works on the current one) */
} na3d_plan_info;

/*
 * na3d_plan - the tiling na3d_fwd would use for this problem, computed on the
 * host without touching a GPU. Arguments as for na3d_fwd; returns the same
 * argument-validation codes (without the pointer, alignment, alias and device
 * checks). `info` must not be NULL.
 */
int na3d_plan(int64_t T, int64_t H, int64_t W, int64_t NH, int64_t HD,
              int64_t KT, int64_t KH, int64_t KW, na3d_plan_info* info);

/*
 * na3d_device_status - after the work already enqueued on `stream`, takes
 * the current device's timeout flag and synchronizes `stream`. The flag is
 * set by any na3d kernel on the device whose pipeline wait gave up (a
 * deadlock guard: each wait inside the kernels is bounded, and a wait that
 * runs out records the flag, drains its in-flight copies and MMAs, frees its
 * tensor memory and returns, leaving part of its output unwritten).
 * "Takes" means read and cleared in one atomic step on the device: each
 * timeout is reported by exactly one call. The flag is per device, not per
 * launch: with several threads or streams launching on one device, the call
 * reports a timeout of any of their launches that completed before it.
 * Returns NA3D_ERR_DEVICE_TIMEOUT if the flag was set, NA3D_ERR_CUDA if the
 * enqueue or the synchronization fails, else NA3D_OK.
 */
int na3d_device_status(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NA3D_H */
