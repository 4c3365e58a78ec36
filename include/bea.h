/*
 * bea.h — C ABI of the blockwise exact attention library (libbea.so).
 *
 * Exact softmax attention computed block by block with an online softmax on
 * one GB300 (sm_103a), its backward pass recomputed from the per-row
 * log-sum-exp, and the log-sum-exp merge that folds a partial (out, lse) from
 * one K/V block into a running (out, lse) — the step ring attention repeats
 * once per K/V rotation.
 *
 * Tensors.
 *   Every tensor is described by a bea_tensor: a DEVICE pointer, a dtype, a
 *   rank, a shape and strides in ELEMENTS. The caller owns every buffer; the
 *   library never allocates, frees or keeps a pointer after a call returns.
 *   Sequence tensors are [n, l, h, d] (batch, sequence, heads, head dim) with
 *   the last dimension contiguous (stride 1), the base pointer 16-byte
 *   aligned and the other strides multiples of 16 bytes, so that chunk views
 *   of a longer sequence (an offset base pointer with the parent's strides)
 *   are accepted without a copy. The log-sum-exp is [n, h, l] fp32, natural
 *   log, softmax_scale included, with a contiguous last dimension and
 *   4-byte alignment
 *   (flash_attn_jax flash_sharding.py, sections "Sharding" and "Ring
 *   Forward": out [n,l,h,d], lse [n,h,l]).
 *
 * Grouped-query attention.
 *   q has h heads, k and v have h_kv heads with h % h_kv == 0; query head i
 *   reads K/V head i / (h / h_kv) (picotron context_parallel.py,
 *   RingAttention._repeat_kv), without expanding K/V in memory.
 *
 * Masks.
 *   is_causal: query i sees key j only if j <= i (picotron
 *   ring_attention_forward: the upper triangle is masked).
 *   window (left, right), -1 meaning unbounded: key j is visible to query i
 *   iff (left < 0 || j >= i - left) && (right < 0 || j <= i + right). The
 *   pages only ever pass (-1, -1); this inclusive reading is the library's.
 *   is_causal forces right = 0; right > 0 together with is_causal is an
 *   argument error.
 *   Positions: the window compares sequence positions, with key j at position
 *   j + key_offset relative to query i at position i. bea_flash_mha_fwd and
 *   bea_flash_mha_bwd use key_offset = lq - lk, which aligns the last query
 *   with the last key (bottom-right; 0 when lq == lk, the only case the pages
 *   use); the fused ring step and the K/V-block stage take it explicitly (a
 *   ring chunk pair passes the distance between its key and query chunks).
 *   Sequence lengths must be below 2^30.
 *   A query row that sees no key gets out = 0 and lse = -inf.
 *
 * Streams and errors.
 *   `stream` is a cudaStream_t (NULL = legacy default stream) of the current
 *   device. Every call validates all arguments on the host first and
 *   launches nothing when a check fails. Launches are asynchronous. Return
 *   values: BEA_OK or one of the negative BEA_ERR_* codes. No kernel traps:
 *   a kernel whose internal wait runs past its time limit ORs a flag into a
 *   per-device status word, which bea_get_device_status() reads.
 *
 * Thread safety: calls may come from several host threads; the library's
 * host state is a per-device cache filled on first use and the one-shot test
 * hook armed by bea_selftest_inject_abort (process-wide: the next launch from
 * any thread takes it).
 */
#ifndef BEA_H_
#define BEA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define BEA_VERSION 1

typedef enum bea_dtype {
  BEA_BF16 = 0, /* bfloat16 */
  BEA_F32 = 1,  /* float32 */
  BEA_I32 = 2   /* int32: lengths, tables, slots and positions of the paged and rotary calls only */
} bea_dtype;

typedef enum bea_status {
  BEA_OK = 0,
  BEA_ERR_ARG = -1,         /* null pointer, bad scalar (scale, window, flags) */
  BEA_ERR_SHAPE = -2,       /* shapes inconsistent with each other */
  BEA_ERR_DTYPE = -3,       /* dtype not allowed for this argument */
  BEA_ERR_ALIGN = -4,       /* pointer or stride not 16-byte aligned, last dim not contiguous */
  BEA_ERR_UNSUPPORTED = -5, /* valid request this build does not implement (e.g. head dim) */
  BEA_ERR_CUDA = -6,        /* a CUDA runtime/driver call failed */
  BEA_ERR_TIMEOUT = -7,     /* a kernel wait ran past its limit (from bea_get_device_status) */
  BEA_ERR_WORKSPACE = -8,   /* workspace missing, misaligned or too small */
  BEA_ERR_PAGES = -9        /* a paged call met a page, slot or length out of range (from bea_get_device_status) */
} bea_status;

typedef struct bea_tensor {
  void* data;        /* device pointer to element [0,0,0,0] */
  int32_t dtype;     /* bea_dtype */
  int32_t ndim;      /* 4 for [n,l,h,d] tensors, 3 for [n,h,l] lse tensors, 1 to 3 for int32 tensors */
  int64_t shape[4];  /* first ndim entries used */
  int64_t stride[4]; /* in elements; first ndim entries used */
} bea_tensor;

/*
 * Forward: out = softmax(softmax_scale * q k^T + mask) v and
 * lse = log(sum_j exp(softmax_scale * q.k_j + mask_j)) per query row
 * (picotron context_parallel.py, ring_attention_forward; flash_attn_jax
 * flash_sharding.py, the local fwd(q, k, v) of partition_fwd).
 *
 *   q    [n, lq, h, d]     bf16 or f32
 *   k, v [n, lk, h_kv, d]  same dtype as q
 *   out  [n, lq, h, d]     bf16 q: bf16 or f32; f32 q: f32 (written)
 *   lse  [n, h, lq]        f32 (written)
 *   softmax_scale must be finite and > 0.
 *   bf16: d must be 64 or 128; runs on the tcgen05 tensor cores with fp32
 *   accumulation (P is rounded to bf16 before P v).
 *   f32: 4 <= d <= 128, d % 4 == 0; runs an exact fp32 SIMT kernel.
 */
int bea_flash_mha_fwd(const bea_tensor* q, const bea_tensor* k, const bea_tensor* v, const bea_tensor* out,
                      const bea_tensor* lse, float softmax_scale, int is_causal, int window_left,
                      int window_right, void* stream);

/*
 * Fused ring step: the forward of one K/V block, folded straight into a
 * running fp32 accumulator by the log-sum-exp merge (flash_attn_jax
 * flash_sharding.py, "Ring Forward": the block's (out, lse) merged into the
 * carried (o, lse) once per ring step). Equal to bea_flash_mha_fwd into a
 * temporary followed by bea_ring_merge, without writing the block's output
 * to memory and without its rounding to bf16.
 *
 *   q, k, v    as for the forward, bf16 only (f32: BEA_ERR_UNSUPPORTED)
 *   out_acc    [n, lq, h, d] f32, read and written
 *   lse_acc    [n, h, lq]    f32, read and written
 *   out_final  NULL, or [n, lq, h, d] bf16: also receives the merged rows cast
 *              to bf16 (the last step of a ring)
 *   key_offset position of key 0 relative to query 0 (see Masks); |key_offset|
 *              <= 2^30
 * Per row, with La the accumulator's and L the block's log-sum-exp:
 * M = max(La, L); if M == -inf the row is left unchanged; otherwise
 * L' = M + log1p(exp(min(La, L) - M)), out_acc <- exp(La - L') out_acc +
 * exp(L - L') O_block, lse_acc <- L'.
 */
int bea_flash_mha_fwd_merge(const bea_tensor* q, const bea_tensor* k, const bea_tensor* v, const bea_tensor* out_acc,
                            const bea_tensor* lse_acc, const bea_tensor* out_final, float softmax_scale, int is_causal,
                            int window_left, int window_right, int64_t key_offset, void* stream);

/*
 * Bytes of device workspace bea_flash_mha_bwd needs for q of shape
 * [n, lq, h, d] (an fp32 dQ accumulator plus two fp32 values per row).
 */
size_t bea_flash_mha_bwd_workspace_size(int64_t n, int64_t lq, int64_t h, int64_t d);

/*
 * Backward from the GIVEN out and lse (picotron context_parallel.py,
 * ring_attention_backward, Steps 1-6):
 *   P = exp(softmax_scale * q k^T - lse) (masked entries 0), dV = P^T dO,
 *   dP = dO v^T, D = rowsum(dO * out), dS = P * (dP - D),
 *   dQ = softmax_scale * dS k, dK = softmax_scale * dS^T q,
 * with dK, dV summed over the query heads of each K/V head. Using the final
 * out/lse of the full row (not a chunk's) is what lets ring chunk pairs add
 * their partial gradients (flash_sharding.py, "Ring Backward").
 *
 *   dout        [n, lq, h, d]    q's dtype
 *   q, k, v     as for the forward
 *   out         [n, lq, h, d]    q's dtype, or f32
 *   lse         [n, h, lq]       f32
 *   dq          [n, lq, h, d]    q's dtype or f32 (written)
 *   dk, dv      [n, lk, h_kv, d] q's dtype or f32 (written)
 *   accumulate  0: dq/dk/dv are overwritten; 1: the gradients are ADDED to
 *               dq/dk/dv, which must then all be f32 (ring chunk pairs).
 *   workspace   device buffer of at least bea_flash_mha_bwd_workspace_size()
 *               bytes, 256-byte aligned, owned by the caller, contents on
 *               entry irrelevant; calls that may run concurrently need
 *               separate workspaces.
 */
int bea_flash_mha_bwd(const bea_tensor* dout, const bea_tensor* q, const bea_tensor* k, const bea_tensor* v,
                      const bea_tensor* out, const bea_tensor* lse, const bea_tensor* dq, const bea_tensor* dk,
                      const bea_tensor* dv, float softmax_scale, int is_causal, int window_left,
                      int window_right, int accumulate, void* workspace, size_t workspace_bytes,
                      void* stream);

/*
 * The bf16 backward in its three stages, for a caller that accumulates the dQ
 * of one set of query rows over several K/V blocks: the backward of ring
 * attention, where each query chunk meets every visible K/V chunk once
 * (flash_attn_jax flash_sharding.py, "Ring Backward": dq accumulates over the
 * steps; picotron context_parallel.py, RingAttentionFunc.backward). Running
 * prepare once, kv_block once per K/V block, then finish once keeps dQ in
 * fp32 in the workspace across blocks and computes D once per query chunk.
 * bea_flash_mha_bwd on bf16 inputs is exactly prepare + kv_block + finish.
 *
 * All three take the same workspace, sized by
 * bea_flash_mha_bwd_workspace_size(n, lq, h, d) of the query-side tensors,
 * 256-byte aligned. Between prepare and finish it holds the state of the
 * accumulation; calls on it must be ordered on one stream. Only bf16 q/k/v
 * are supported (f32 inputs: BEA_ERR_UNSUPPORTED; use bea_flash_mha_bwd).
 *
 * prepare  (Step "D = rowsum(dO * O)"): dout [n, lq, h, d] bf16;
 *          out same shape, bf16 or f32; lse [n, h, lq] f32. Writes D and
 *          lse * log2(e) per row and zeroes the fp32 dQ accumulator.
 * kv_block (Steps P, dV, dP, dS, dK, and dQ's sum over these keys): dout,
 *          q [n, lq, h, d] bf16, k, v [n, lk, h_kv, d] bf16; dk, dv
 *          [n, lk, h_kv, d] bf16 or f32, written (accumulate 0) or added to
 *          (accumulate 1, both f32). Adds this block's dS k into the
 *          accumulator. The mask arguments are those of bea_flash_mha_bwd,
 *          with key_offset the position of this block's key 0 relative to
 *          query 0 (see Masks).
 * finish   dq [n, lq, h, d] bf16 or f32: dq = softmax_scale * accumulator,
 *          written (accumulate 0) or added to an f32 dq (accumulate 1).
 */
int bea_flash_mha_bwd_prepare(const bea_tensor* dout, const bea_tensor* out, const bea_tensor* lse,
                              void* workspace, size_t workspace_bytes, void* stream);
int bea_flash_mha_bwd_kv_block(const bea_tensor* dout, const bea_tensor* q, const bea_tensor* k,
                               const bea_tensor* v, const bea_tensor* dk, const bea_tensor* dv,
                               float softmax_scale, int is_causal, int window_left, int window_right,
                               int64_t key_offset, int accumulate, void* workspace, size_t workspace_bytes,
                               void* stream);
int bea_flash_mha_bwd_finish(const bea_tensor* dq, float softmax_scale, int accumulate, void* workspace,
                             size_t workspace_bytes, void* stream);

/*
 * Ring attention replayed on one GPU in one call (flash_attn_jax
 * flash_sharding.py, "Ring Forward"): the sequence is split into n_chunks
 * equal chunks; at ring step t query chunk i meets the K/V chunk
 * (i - t) mod n_chunks (the chunk that started on device i - t when K/V move
 * i -> i+1), and every live pair's (out, lse) is folded into the running
 * fp32 (out_acc, lse) by the log-sum-exp merge of bea_flash_mha_fwd_merge.
 * Pairs whose keys are all masked (under is_causal every pair above the
 * diagonal; under a window every pair beyond it) are skipped; the window
 * compares sequence positions, so a chunk pair sees exactly the keys the
 * single call would. All pairs of one ring step run as one launch over chunk
 * views; the launches of one call are chained on `stream` by programmatic
 * dependent launch (a step starts computing while the step before finishes
 * and merges only after it has).
 *
 *   q          [n, l, h, d] bf16; k, v [n, l, h_kv, d] bf16 (same l)
 *   out_acc    [n, l, h, d] f32, written: the result (the ring's accumulator)
 *   lse        [n, h, l] f32, written
 *   out_final  NULL, or [n, l, h, d] bf16: also receives the result cast to
 *              bf16, written at each query chunk's last live step
 *   n_chunks   >= 1, dividing l
 * Errors as for bea_flash_mha_fwd; l % n_chunks != 0 is BEA_ERR_ARG, f32
 * inputs BEA_ERR_UNSUPPORTED.
 */
int bea_ring_attention_fwd(const bea_tensor* q, const bea_tensor* k, const bea_tensor* v, const bea_tensor* out_acc,
                           const bea_tensor* lse, const bea_tensor* out_final, int n_chunks, float softmax_scale,
                           int is_causal, int window_left, int window_right, void* stream);

/*
 * Workspace bytes of bea_ring_attention_bwd for q [n, l, h, d] split into
 * n_chunks chunks (0 when n_chunks does not divide l).
 */
size_t bea_ring_attention_bwd_workspace_size(int64_t n, int64_t l, int64_t h, int64_t d, int n_chunks);

/*
 * Backward of ring attention on one GPU in one call (flash_attn_jax
 * flash_sharding.py, "Ring Backward"; picotron context_parallel.py,
 * RingAttentionFunc.backward): every live chunk pair (same schedule and masks
 * as bea_ring_attention_fwd) is differentiated once with the FINAL out/lse of
 * its query rows, and the partial gradients are summed in fp32: dQ of a query
 * chunk in the workspace accumulator, dK/dV of a key chunk in place. All
 * pairs of one ring step run as one launch; per batch row: one preprocess,
 * one launch per live step, one dQ conversion.
 *
 *   dout, q    [n, l, h, d] bf16; k, v [n, l, h_kv, d] bf16
 *   out        [n, l, h, d] bf16 or f32; lse [n, h, l] f32
 *   dq         [n, l, h, d] f32, written; dk, dv [n, l, h_kv, d] f32, written
 *   workspace  >= bea_ring_attention_bwd_workspace_size() bytes, 256-byte
 *              aligned, caller-owned, contents on entry irrelevant
 */
int bea_ring_attention_bwd(const bea_tensor* dout, const bea_tensor* q, const bea_tensor* k, const bea_tensor* v,
                           const bea_tensor* out, const bea_tensor* lse, const bea_tensor* dq, const bea_tensor* dk,
                           const bea_tensor* dv, int n_chunks, float softmax_scale, int is_causal, int window_left,
                           int window_right, void* workspace, size_t workspace_bytes, void* stream);

/*
 * bea_flash_mha_bwd without a caller-supplied workspace. (The pages have no
 * counterpart; this is a library convenience.)
 *
 * For callers that cannot allocate device memory: code that reaches the
 * library only through a C function pointer from another language or plugin
 * host that hands over just the tensors it owns, or a long-running serving
 * loop that must not call cudaMalloc (which can synchronise the device). The
 * workspace comes from a fixed array of BEA_NOALLOC_BWD_SCRATCH_BYTES in the
 * library's own device memory; every GPU that loads the library holds that
 * array until the process exits. This call allocates nothing.
 *
 * Arguments and results are those of bea_flash_mha_bwd, checked in the same
 * order and with the same error codes. Only a call that passes those checks
 * and whose workspace (bea_flash_mha_bwd_workspace_size, computed without
 * overflow) exceeds the array returns BEA_ERR_WORKSPACE, before anything is
 * launched.
 *
 * The first call in a device's context looks up the array's device address
 * (cudaGetSymbolAddress) with that device current and caches it for that
 * context; a new context on the device (e.g. after cudaDeviceReset) looks it
 * up again on its first call. Make that first call before any stream
 * capture. All calls on a device share the one
 * array, so two calls whose kernels may overlap on the GPU (different
 * streams, or several host threads) race on it: order them on one stream.
 * The array keeps the last call's contents; each call rewrites all of it
 * that it reads, so nothing needs clearing between calls.
 */
#define BEA_NOALLOC_BWD_SCRATCH_BYTES (64u * 1024u * 1024u)
int bea_flash_mha_bwd_noalloc(const bea_tensor* dout, const bea_tensor* q, const bea_tensor* k,
                              const bea_tensor* v, const bea_tensor* out, const bea_tensor* lse,
                              const bea_tensor* dq, const bea_tensor* dk, const bea_tensor* dv,
                              float softmax_scale, int is_causal, int window_left, int window_right,
                              int accumulate, void* stream);

/*
 * Log-sum-exp merge, in place on the accumulator (flash_attn_jax
 * flash_sharding.py, "Ring Forward"; the same fold as picotron
 * update_out_and_lse in its sigmoid form). Per row r = (b, i, head):
 *   M = max(La, Lb); if M == -inf the row is left unchanged; otherwise
 *   L = M + log1p(exp(min(La, Lb) - M)), Oa <- exp(La - L) Oa + exp(Lb - L) Ob,
 *   La <- L.
 *
 *   out_acc   [n, l, h, d] f32 (read and written)
 *   lse_acc   [n, h, l]    f32 (read and written)
 *   out_blk   [n, l, h, d] bf16 or f32
 *   lse_blk   [n, h, l]    f32
 *   out_final NULL, or [n, l, h, d] bf16: also receives the merged rows cast
 *             to bf16 (the last step of a ring).
 *   d must be 16, 32, 64 or 128.
 */
int bea_ring_merge(const bea_tensor* out_acc, const bea_tensor* lse_acc, const bea_tensor* out_blk,
                   const bea_tensor* lse_blk, const bea_tensor* out_final, void* stream);

/*
 * Rotary positions with one or several axes (time, height, width ...), q and k
 * in one launch. Pair p of a row is (x_p, x_{p + d/2}), the rotate-half pairs;
 * its angle at batch b, position i is
 *   angle = positions[axis_of_pair[p], b, i] * freq[p]
 * and y_p = x_p cos - x_{p+d/2} sin, y_{p+d/2} = x_{p+d/2} cos + x_p sin. With
 * `inverse` the angle is negated: the rotation's adjoint, hence its gradient
 * (dx from dy), and its inverse.
 *
 *   q          [n, l, h, d]    bf16 or f32
 *   k          NULL, or [n, l, h_k, d], q's dtype
 *   positions  [axes, n, l]    i32, any sign, 1 <= axes <= 8; outer strides may
 *              be 0 (one row of positions for the whole batch)
 *   axis_of_pair, freq   HOST arrays of d/2 entries: axis index in [0, axes)
 *              and radians per position (finite); read during the call only
 *   q_out, k_out   shapes and dtype of q, k (written); k_out NULL iff k is.
 *              Each may be its input itself (same pointer, same strides), and
 *              must not overlap the inputs otherwise; not broadcast.
 *   d: bf16 a multiple of 16, f32 a multiple of 8, at most 256.
 * The angle is reduced modulo a whole turn in 64-bit fixed point, with the turns
 * per position held as a multiple of 2^-64: it is off by at most |position| *
 * (2^-65 + 2^-52 * |freq| / (2 pi)) turns, so a far position loses next to
 * nothing. Less its nearest quarter turn it is rounded to fp32, off by at most
 * 2^-28 turns. Cosine and sine are then within 2^-23.5 of the true ones; products
 * in fp32, one rounding.
 */
int bea_rope_axes(const bea_tensor* q, const bea_tensor* k, const bea_tensor* positions, const int32_t* axis_of_pair,
                  const double* freq, int inverse, const bea_tensor* q_out, const bea_tensor* k_out, void* stream);

/*
 * The rotation of bea_rope_axes with its other layouts, and the RMS norm that
 * some models put before it, q and k in one launch. Of a row x (d elements):
 *   norm 1: y = w * x / sqrt(mean(x^2) + eps), w the row of weights; norm 0: y = x
 *   pair p < pairs is (y_p, y_{p + pairs}), or, interleaved, (y_{2p}, y_{2p + 1});
 *   (a, b) becomes amplitude * (a cos - b sin, b cos + a sin), the angle as for
 *   bea_rope_axes; what lies behind the 2 * pairs first elements is not turned.
 *
 *   q, k, positions, axis_of_pair, freq, q_out, k_out  as for bea_rope_axes, the
 *              arrays of `pairs` entries (NULL where that is 0)
 *   pairs      0 <= 2 * pairs <= d; not interleaved: a multiple of 8 (bf16) or 4
 *              (f32), else BEA_ERR_UNSUPPORTED
 *   amplitude  finite
 *   inverse    1 (norm 0 only): the angles negated, which is the adjoint (and, at
 *              amplitude 1, the inverse)
 *   q_weight, k_weight   NULL (ones) or [d], bf16 or f32 whatever q is; norm 0: NULL
 *   eps        >= 0, finite
 * In fp32, rounded once. d as for bea_rope_axes.
 */
int bea_norm_rope_axes(const bea_tensor* q, const bea_tensor* k, const bea_tensor* positions,
                       const int32_t* axis_of_pair, const double* freq, int pairs, int interleaved, float amplitude,
                       int inverse, const bea_tensor* q_weight, const bea_tensor* k_weight, int norm, float eps,
                       const bea_tensor* q_out, const bea_tensor* k_out, void* stream);

/*
 * The gradient of bea_norm_rope_axes with norm 1: from x (q, k) and the outputs'
 * gradients those of x and of the weights (their sums over all rows in fp32, in a
 * fixed order).
 *   dq_out, dk_out   shapes and dtype of q, k
 *   dq, dk           the same (written); dk, dk_out NULL iff k is. Each may be
 *                    the output's gradient itself (same pointer, same strides).
 *   dq_weight, dk_weight   NULL (not wanted), or [d] of the weight's dtype (written)
 *   workspace        bea_norm_rope_axes_bwd_workspace_size(d) bytes, 256-byte
 *                    aligned; may be NULL where no weight's gradient is wanted.
 *                    Contents on entry irrelevant; calls that may run
 *                    concurrently need separate workspaces.
 */
size_t bea_norm_rope_axes_bwd_workspace_size(int64_t d);
int bea_norm_rope_axes_bwd(const bea_tensor* q, const bea_tensor* k, const bea_tensor* dq_out, const bea_tensor* dk_out,
                           const bea_tensor* positions, const int32_t* axis_of_pair, const double* freq, int pairs,
                           int interleaved, float amplitude, const bea_tensor* q_weight, const bea_tensor* k_weight,
                           float eps, const bea_tensor* dq, const bea_tensor* dk, const bea_tensor* dq_weight,
                           const bea_tensor* dk_weight, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Paged K/V cache. A cache is [num_pages, page_size, h_kv, d] (any 16-byte
 * aligned outer strides, so a [num_pages, h_kv, page_size, d] cache is passed
 * as its permuted view). Request r owns the pages block_table[r, 0 ..
 * ceil(len_r / page_size)), and its token at position p lives in page
 * block_table[r, p / page_size] at offset p % page_size; its SLOT is page *
 * page_size + offset. Free pages are a stack: free_pages[0 .. n_free), the top
 * at n_free - 1. For reading (bea_paged_decode) pages may be shared between rows
 * of a table. bea_paged_plan takes every page to be owned by one row: it does
 * not count owners, so a row whose pages another row shares has to be kept from
 * ending (or the shared entries taken out of one of the two) by the caller, and
 * a row may not add tokens to a last page that it shares.
 *
 * What the device finds out of range (a length beyond the table, a page or a
 * slot outside the cache) is never accessed: it is left out as described at
 * each call, and bea_get_device_status then reads BEA_ERR_PAGES.
 */

/*
 * One scheduling step of a paged cache from request lengths, on the GPU: ends
 * requests, hands pages to the tokens that are added, and lists where those
 * tokens go.
 *
 *   lens        [n] i32   tokens request r holds now
 *   new_lens    [n] i32   tokens it adds (>= 0), or -1: the request ends
 *   block_table [n, max_pages] i32, read and written: entries of new pages
 *   free_pages  [F] i32, read and written: the stack; ended requests' pages are
 *               pushed in row order, a row's pages in table order; then new
 *               pages are popped in row order
 *   n_free      [1] i32   height of the stack
 *   slot_map    [capacity] i32, written: the slot of every added token, requests
 *               in row order, tokens in sequence order; -1 behind the last
 *   positions   [capacity] i32, written: each added token's position in its
 *               request; 0 behind the last
 *   cu_new      [n + 1] i32, written: added tokens before row r; [n] is their number
 *   cu_pages    [n + 1] i32, written: pages popped before row r
 *   lens_out    [n] i32, written: the new lengths (0 for ended requests); may be `lens`
 *   n_free_out  [1] i32, written; may be `n_free`
 * All or nothing: if a length or new length is negative (other than -1 as new
 * length) or passes max_pages * page_size, if the added tokens pass the
 * capacity, or if the stack would run empty or pass F, the step changes
 * nothing (lens_out = lens, n_free_out = n_free, slot_map all -1, positions
 * and the cu arrays all 0) and the device status reads BEA_ERR_PAGES. A slot
 * that is not in [0, 2^31) is written as -1, with the same status.
 * No two arrays may overlap other than as said. page_size in [1, 2^20].
 */
int bea_paged_plan(const bea_tensor* lens, const bea_tensor* new_lens, const bea_tensor* block_table,
                   const bea_tensor* free_pages, const bea_tensor* n_free, int64_t page_size,
                   const bea_tensor* slot_map, const bea_tensor* positions, const bea_tensor* cu_new,
                   const bea_tensor* cu_pages, const bea_tensor* lens_out, const bea_tensor* n_free_out,
                   void* stream);

/*
 * Writes new keys and values into a paged cache: token t (t = i * l + j for
 * k[i, j]) goes to slot slot_map[t].
 *
 *   k, v              [n, l, h_kv, d] bf16 or f32
 *   slot_map          [n * l] i32; -1: the token is not written. Two tokens must
 *                     not have the same slot (which of them stays would depend
 *                     on timing, 16 bytes at a time).
 *   k_cache, v_cache  [num_pages, page_size, h_kv, d], k's dtype (written); same
 *                     shape, own strides; num_pages * page_size < 2^31
 *   d * element size must be a multiple of 16 bytes.
 * A slot below -1 or past the cache is skipped and reported.
 */
int bea_paged_write(const bea_tensor* k, const bea_tensor* v, const bea_tensor* slot_map, const bea_tensor* k_cache,
                    const bea_tensor* v_cache, void* stream);

/*
 * Attention of one new token per request over a paged cache: the forward of
 * this library for lq = 1, with keys and values read through the block table.
 * The new token is the request's last key (write it first): with len =
 * lens[r], query r sees the keys j with j >= len - 1 - window_left (all of
 * them for window_left = -1) and j < len.
 *
 *   q                 [n, 1, h, d]  bf16 (d 64 or 128) or f32 (4 <= d <= 128, d % 4 == 0)
 *   k_cache, v_cache  [num_pages, page_size, h_kv, d], q's dtype, h % h_kv == 0;
 *                     same shape, own strides
 *   block_table       [n, max_pages] i32, outer stride any
 *   lens              [n] i32
 *   out               [n, 1, h, d]  bf16 q: bf16 or f32; f32 q: f32 (written)
 *   lse               [n, h, 1]     f32, natural log, scale included (written)
 *   workspace         bea_paged_decode_workspace_size() bytes, 256-byte aligned;
 *                     may be NULL when that is 0. Contents on entry irrelevant;
 *                     calls that may run concurrently need separate workspaces.
 * A request of length 0 gets out = 0 and lse = -inf. A length past max_pages *
 * page_size counts as that, a negative one as 0, and the keys of a page
 * outside the cache as masked; each is reported. num_pages * page_size < 2^31;
 * max_pages * page_size < 2^30, and (max_pages * page_size / 8 + 4) * h_kv < 2^31
 * is always enough for the kernels' 32-bit counts (BEA_ERR_SHAPE past them).
 */
size_t bea_paged_decode_workspace_size(int64_t h, int64_t h_kv, int64_t d, int64_t max_keys);
int bea_paged_decode(const bea_tensor* q, const bea_tensor* k_cache, const bea_tensor* v_cache,
                     const bea_tensor* block_table, const bea_tensor* lens, const bea_tensor* out,
                     const bea_tensor* lse, float softmax_scale, int window_left, void* workspace,
                     size_t workspace_bytes, void* stream);

/*
 * bea_paged_decode for groups of requests whose first keys are the same (a
 * prompt that many requests start from): those are read once for the group.
 *
 *   q, k_cache, v_cache, block_table, lens, out, lse   as for bea_paged_decode,
 *               bf16 (f32: BEA_ERR_UNSUPPORTED); no window
 *   group_rows  [groups + 1] i32, ascending: group g is the rows group_rows[g] ..
 *               group_rows[g + 1] - 1; rows of no group share nothing
 *   shared_lens [groups] i32: the group's first shared_lens[g] keys are the same
 *               for all its requests, that is, the rows of the table name the same
 *               pages for them (bea_paged_fork makes such rows). The first row that
 *               holds a request is read for all whose tables name its pages; a row
 *               that names another one among them is read for itself. (Where that is
 *               the last of them only, as in forks of a prompt that ends inside a
 *               page, that page is not shared.)
 *   workspace   bea_paged_decode_shared_workspace_size() bytes, 256-byte aligned;
 *               may be NULL when that is 0. Contents on entry irrelevant; calls that may run concurrently need
 *               separate workspaces.
 * A request of length 0 takes no part in its group, and gets out = 0, lse =
 * -inf. Shared is what is whole tiles of 128 keys of the shortest request's and
 * in pages of the cache; what is left over is read for each request. Where the
 * table has no room for 96 MB of keys and values that sharing could save, the
 * groups are not looked at: the call is bea_paged_decode, which is then faster.
 * groups <= 1024. Results are those of bea_paged_decode up to rounding: in the
 * product with the values weights of the shared keys have 16 bits, and an f32 out is
 * within 2^-14 of sum(p |v|), however many they are. group_rows out of order or
 * range: nothing is shared, and reported; a negative shared_lens counts as 0 and is
 * reported; the rest as bea_paged_decode reports it. (2 h n + 40960 <
 * 2^31, and h_kv (n h / h_kv / 256 + min(groups, n)) (max_keys / 128 + 6) < 2^31, else
 * BEA_ERR_SHAPE.)
 */
size_t bea_paged_decode_shared_workspace_size(int64_t n, int64_t h, int64_t h_kv, int64_t d, int64_t max_keys,
                                              int64_t groups);
int bea_paged_decode_shared(const bea_tensor* q, const bea_tensor* k_cache, const bea_tensor* v_cache,
                            const bea_tensor* block_table, const bea_tensor* lens, const bea_tensor* group_rows,
                            const bea_tensor* shared_lens, const bea_tensor* out, const bea_tensor* lse,
                            float softmax_scale, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Pages that several rows of a table hold. shares[p] is the number of rows that
 * hold page p beyond the first: 0 for a page of one row, and for a free one.
 * bea_paged_plan neither reads nor changes it (the pages that it hands out have
 * 0), but it takes every page to be owned by one row: rows of a table with
 * shared pages are ended by bea_paged_free, before the plan, which then meets
 * them with length 0.
 *
 * Outputs may be their inputs (lens_out = lens, n_free_out = n_free, shares_out =
 * shares); no arrays overlap otherwise.
 *
 * bea_paged_fork: rows begin as copies of other rows, sharing their pages.
 *   src         [n] i32   -1: row r takes no part; else it becomes a fork of row
 *               src[r], which does not fork itself. Row r has to be free (length 0).
 *   tokens      NULL, or [n] i32: the row takes the source's first tokens[r]
 *               tokens; -1 (and NULL): all of them
 *   lens, block_table (read and written), free_pages, n_free   as for
 *               bea_paged_plan; free_pages is only read
 *   shares      [num_pages] i32
 *   lens_out [n], n_free_out [1], shares_out [num_pages]   written
 *   copies      [n, 3] i32, written: where a fork ends inside a page that page's
 *               tokens are copied to a page of its own, popped in row order: (page,
 *               new page, tokens); (-1, -1, 0) for a fork that needs none, (-1, -1,
 *               -1) for other rows. For bea_paged_copy, in every layer.
 * Full pages are shared. All or nothing: a row or a number out of range, a
 * source that forks, a row that is not free, a length beyond the table, or a
 * stack that runs empty leaves everything as it is (every copy -1) and the device
 * status reads BEA_ERR_PAGES. A page outside [0, num_pages) in a source's row is
 * handed on uncounted, and not copied; it is reported.
 */
int bea_paged_fork(const bea_tensor* src, const bea_tensor* tokens, const bea_tensor* lens,
                   const bea_tensor* block_table, const bea_tensor* shares, const bea_tensor* free_pages,
                   const bea_tensor* n_free, int64_t page_size, const bea_tensor* lens_out,
                   const bea_tensor* n_free_out, const bea_tensor* shares_out, const bea_tensor* copies, void* stream);

/*
 * Rows end; pages that no row holds any more go back on the stack, in ascending
 * order of their ids.
 *   ends        [n] i32: row r ends where it is negative (the new_lens of
 *               bea_paged_plan can be passed)
 *   free_pages  read and written; the rest as for bea_paged_fork
 *   lens_out    0 for the rows that end
 * A height of the stack out of range leaves everything as it is; a row whose
 * length is out of range stays; pages outside [0, num_pages) are passed over;
 * pages that pass the stack's end are lost; a page given back more often than it
 * was held goes on the stack once. Each is reported.
 */
int bea_paged_free(const bea_tensor* ends, const bea_tensor* lens, const bea_tensor* block_table,
                   const bea_tensor* shares, const bea_tensor* free_pages, const bea_tensor* n_free, int64_t page_size,
                   const bea_tensor* lens_out, const bea_tensor* n_free_out, const bea_tensor* shares_out,
                   void* stream);

/*
 * Used pages move to the lower end of the cache: the lowest free page takes the
 * highest used one's place, the next the next, as long as that is a move
 * downwards and `copies` has room. All pages that are not on the stack count as
 * used.
 *   lens [n], block_table [n, max_pages], shares [num_pages], free_pages [F],
 *   n_free [1]         read
 *   block_table_out    the table with the new pages; entries behind a row's last
 *                      page are those of the table
 *   shares_out, free_pages_out (the lowest page on top, -1 behind the last; the
 *                      height stays)
 *   page_map           [num_pages] i32: where each page went, itself if nowhere
 *   copies             [capacity, 3] i32: (page, new page, page_size) of every
 *                      move, then -1
 * block_table_out may be block_table, free_pages_out free_pages and shares_out
 * shares. The moves' contents are copied by bea_paged_copy, before anything
 * else writes the cache. num_pages <= 2^20. A stack with a page twice, a page
 * outside [0, num_pages) or a height out of range: nothing moves; a table entry
 * outside stays as it is, a length out of range counts as 0 or all of the table.
 * Each is reported.
 */
int bea_paged_compact(const bea_tensor* lens, const bea_tensor* block_table, const bea_tensor* shares,
                      const bea_tensor* free_pages, const bea_tensor* n_free, int64_t page_size,
                      const bea_tensor* block_table_out, const bea_tensor* shares_out, const bea_tensor* free_pages_out,
                      const bea_tensor* page_map, const bea_tensor* copies, void* stream);

/*
 * Copies the first tokens of pages to other pages, in every cache alike.
 *   copies     [m, 3] i32, rows one behind the other: (page, new page, tokens);
 *              tokens <= 0: no copy. No new page may be a page of another copy.
 *   caches     HOST array of n_caches tensors [num_pages, page_size, h_kv, d]
 *              (keys and values of every layer), bf16 or f32, one shape, own
 *              strides, none overlapping; read during the call only
 * d * element size must be a multiple of 16 bytes. A copy with a page outside the
 * cache, from a page to itself, or of more than page_size tokens is left out and
 * reported.
 */
int bea_paged_copy(const bea_tensor* copies, const bea_tensor* caches, int n_caches, void* stream);

/*
 * Synchronises `stream`, reads the device status word of the current device
 * and clears it. Returns BEA_OK, BEA_ERR_TIMEOUT if any kernel since the last
 * read gave up a wait, BEA_ERR_UNSUPPORTED if a kernel met a configuration it
 * cannot run, BEA_ERR_PAGES if a paged call met a page, slot or length out of
 * range, or BEA_ERR_CUDA.
 */
int bea_get_device_status(void* stream);

/* Static English text for a status code. */
const char* bea_status_string(int code);

/* BEA_VERSION of the built library. */
int bea_version(void);

/*
 * Failure-detection self test: launches one CTA whose thread waits on an
 * mbarrier that nothing arrives on, with a limit of `limit_us` microseconds
 * (1..2000000). The wait gives up, the kernel returns normally and the
 * status word reads BEA_ERR_TIMEOUT afterwards. No trap, no fault.
 */
int bea_selftest_wait_timeout(int limit_us, void* stream);

/*
 * Failure-detection self test of the attention kernels. Arms a one-shot
 * injection: the next bf16 forward or backward main-kernel launch of this
 * process (bea_flash_mha_fwd, _fwd_merge, _bwd, _bwd_kv_block, _bwd_noalloc)
 * behaves in its first CTA as if a wait of the MMA-issuing warp had run out of
 * time at tile (forward) or iteration (backward) `tile`. That CTA raises its
 * abort flag and records BEA_STATUS_TIMEOUT. Every other role of the CTA then
 * leaves its loop on its next wait, in-flight copies land, TMEM is freed and
 * the kernel returns normally. The outputs of that launch are undefined; the
 * status word reads BEA_ERR_TIMEOUT afterwards. `tile` = -1 disarms.
 * Returns BEA_ERR_ARG for tile < -1. Nothing traps or faults.
 */
int bea_selftest_inject_abort(int tile);

/* Number of kernels the last successful call on this host thread launched. */
int bea_last_launch_count(void);

#ifdef __cplusplus
}
#endif

#endif /* BEA_H_ */
