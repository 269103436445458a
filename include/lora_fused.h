/*
 * lora_fused.h -- C ABI of the MI355X (gfx950) LoRA linear layer.
 *
 * The layer (page "LoRAFusion: Efficient LoRA Fine-Tuning for LLMs", juhe.plus
 * blog, section 2, formula Y = XW + alpha*(XA)B = XW + alpha*S*B; the
 * papers.chlience.com notes, section 3, write the intermediate as S = X^ A with
 * X^ the dropped-out input):
 *
 *     keep = [u16(seed, offset + i*k + j) >= T],  T = floor(p*65536 + 0.5)
 *     S    = s * (keep (.) X) A,                  s = 1/(1-p)
 *     Y    = X W + alpha * S B
 *
 * and its backward with W frozen (no dW; juhe.plus blog, section 2):
 *
 *     dB = alpha * S^T dY      dS = alpha * dY B^T
 *     dA = s * (keep (.) X)^T dS
 *     dX = dY W^T + s * keep (.) (dS A^T)
 *
 * The multi-adapter entry points apply the same maths per token segment with
 * that segment's adapter (papers.chlience.com notes, section 5
 * "FusedMultiLoRA": every input tile carries an adapter id with its rank,
 * scaling factor and dropout ratio, and backward routes gradients to each
 * adapter).
 *
 * Shapes and layouts (all row-major, contiguous):
 *   X  m x k bf16      W  k x n bf16 (frozen)   A  k x r bf16   B  r x n bf16
 *   Y  m x n bf16      dY m x n bf16            dX m x k bf16
 *   dA k x r bf16      dB r x n bf16            (gradients are overwritten)
 *   S  m x r_s fp32    (r_s = r for the single-adapter calls, r_max for the
 *                       multi-adapter calls; columns past a row's rank are 0)
 *   keep_bits          m rows x ceil(k/32) uint32 words; element (i, j) is bit
 *                      j % 32 of word i*ceil(k/32) + j/32; bits past k are 0.
 *
 * The dropout uniform u16(seed, c) of element counter c is 16-bit half
 * (c mod 8) -- low half of the lowest word first -- of the 128-bit output of
 * Philox4x32-10 (Salmon et al., SC'11) under key (seed_lo, seed_hi) and
 * counter (b_lo, b_hi, 0, 0), b = c >> 3.  Counters use the global row index
 * of the call plus `offset`, so a call on rows [r0, r1) of a larger batch with
 * offset + r0*k reproduces those rows exactly.
 *
 * Ownership: every pointer is a caller-owned device buffer (except the few
 * host-side helpers marked "host").  The library never allocates, frees or
 * keeps a pointer past the call.  S and keep_bits are written by the forward
 * call and must stay alive and unchanged until the matching backward call.
 * Scratch space is the caller-provided `workspace`, sized by the matching
 * *_workspace_size() query; it holds nothing between calls.
 *
 * Execution: every entry point only enqueues kernels on `stream` (0 = the
 * default stream) and returns; there is no host synchronisation.  Results
 * are deterministic: the same inputs give bitwise-identical outputs.
 *
 * Errors: arguments are checked on the host before anything is enqueued; on
 * failure nothing is enqueued and a negative lora_status is returned, with
 * detail in lora_last_error_message() (thread-local).  Checks: non-NULL
 * pointers; 16-byte alignment of X, W, Y, dY, dX and the workspace; 4-byte
 * alignment of S and keep_bits; 0 <= m < 2^31; 0 < k, n < 2^31 with
 * k % 8 == 0 and n % 8 == 0; 1 <= r <= 256; 0 <= p < 1; offset % 8 == 0;
 * workspace large enough (LORA_ERR_INVALID_ARG / LORA_ERR_WORKSPACE).  The
 * layer calls (forward and backward) return LORA_ERR_UNSUPPORTED when B
 * (r or r_max by n bf16) or A (k by r or r_max bf16) exceeds 2 GiB, and the
 * backward calls also when k >= 2^25 (their workspace queries are then 0).
 * Products over a bf16 or an expanded W take tiles of less than 2 GiB: 256 rows
 * (all, if there are fewer) of X, Y, dY and dX, of W 64 in a forward and 256
 * for dX; larger ones are LORA_ERR_UNSUPPORTED too.
 * When m == 0 the m-sized buffers (X, Y, S, keep_bits, dY, dX) may be NULL.
 * The multi-adapter tables live in device memory and are never read on the
 * host: an invalid table (segments not ordered, not
 * covering [0, m), adapter index out of range, adapter rank > r_max) gives
 * undefined values in the affected rows but never an out-of-bounds access;
 * multi_lora_check_segments() validates a host copy for callers who want it.
 */
#ifndef LORA_FUSED_H
#define LORA_FUSED_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    LORA_OK = 0,
    LORA_ERR_INVALID_ARG = -1,
    LORA_ERR_UNSUPPORTED = -2,
    LORA_ERR_WORKSPACE = -3,
    LORA_ERR_HIP = -4
} lora_status;

/* One adapter of the multi-adapter calls.  An array of these lives in device
 * memory (papers.chlience.com notes, section 5: the kernel looks up each
 * tile's adapter A, B, rank, scaling factor and dropout ratio from a table).
 * A: k x r, B: r x n, dA: k x r, dB: r x n, all bf16 device pointers.
 * dA/dB are only used by multi_lora_linear_bwd (may be NULL for forward). */
typedef struct {
    const void *A;
    const void *B;
    void *dA;
    void *dB;
    int32_t r;
    float alpha;
    float p;
    int32_t reserved;
} lora_adapter;

/* ---- single adapter (FusedLoRA) ---------------------------------------- */

/* Bytes of workspace lora_linear_fwd needs for this shape (may be 0). */
size_t lora_linear_fwd_workspace_size(int64_t m, int64_t k, int64_t n, int32_t r);

/* Forward: writes Y, S (m x r fp32) and keep_bits.  keep_bits may be NULL
 * only when p == 0 (then every element is kept and no mask is stored).
 * Kernel split (juhe.plus blog, section 4.1, forward items 1 and 2): one
 * kernel streams X once, generating the mask and S = s*(keep (.) X)A; one MFMA
 * GEMM computes XW and adds alpha*S*B before the single write of Y. */
lora_status lora_linear_fwd(const void *X, const void *W, const void *A, const void *B,
                            int64_t m, int64_t k, int64_t n, int32_t r, float alpha, float p,
                            uint64_t seed, uint64_t offset,
                            void *Y, float *S, uint32_t *keep_bits,
                            void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Forward at p = 0 in the concatenated form (FALQON notes, section 5.2, the
 * adapter's down-projection A stacked beside the frozen W as one operand; the
 * recompute-versus-split question of the juhe.plus blog, section 4.1):
 * Y = X W + alpha (X A) B and S = X A (fp32, m x r, row-major) in one GEMM
 * launch.  Each 256 x 256 output tile forms, inside its own K loop, the
 * 256 x r block of S its rows need (A's rows ride along with W's in every
 * stage; about 6% more matrix-core work), then adds alpha S B before the
 * single write of Y: no separate pass over X and no second pass over Y.  The
 * tiles of the first column block also write S, which lora_linear_bwd takes
 * with keep_bits = NULL and p = 0.  Needs no workspace.  r must be 8 or 16
 * and A, B and S 16-byte aligned (else LORA_ERR_UNSUPPORTED; the general
 * forward with p = 0 covers every other case).  Shapes and the other
 * pointers as for lora_linear_fwd; m == 0 returns at once. */
lora_status lora_linear_fwd_concat(const void *X, const void *W, const void *A, const void *B,
                                   int64_t m, int64_t k, int64_t n, int32_t r, float alpha,
                                   void *Y, float *S, hipStream_t stream);

/* Bytes of workspace lora_linear_bwd needs for this shape. */
size_t lora_linear_bwd_workspace_size(int64_t m, int64_t k, int64_t n, int32_t r);

/* Backward: given dY and the forward's S and keep_bits (NULL iff p == 0),
 * writes dX (m x k), dA (k x r) and dB (r x n).  Kernel split (juhe.plus
 * blog, section 4.1, backward items 3 and 5): one pass over dY yields dS and
 * dB; one pass over X and the mask yields dA; an MFMA GEMM computes dY W^T
 * and adds the masked s*(dS A^T) before the single write of dX.  m == 0
 * writes zero dA and dB.  dX may be NULL: the input gradient is then not
 * computed (its GEMM is skipped), e.g. for a layer whose input needs none. */
lora_status lora_linear_bwd(const void *dY, const void *X, const void *W, const void *A,
                            const void *B, const float *S, const uint32_t *keep_bits,
                            int64_t m, int64_t k, int64_t n, int32_t r, float alpha, float p,
                            void *dX, void *dA, void *dB,
                            void *workspace, size_t workspace_bytes, hipStream_t stream);

/* The same backward for callers that cannot allocate device memory (code
 * under graph capture, tight training loops, harnesses that forbid
 * allocation): it takes no workspace and uses a scratch array of
 * lora_linear_bwd_noalloc_max_scratch() bytes (64 MiB) that the library holds
 * in static device memory, one per GPU, until the process ends.  It never
 * allocates or frees.  The scratch of the current device is used (the stream
 * must belong to it).  A shape whose workspace (lora_linear_bwd_workspace_size)
 * exceeds the scratch returns LORA_ERR_UNSUPPORTED before anything is
 * enqueued.  Every call on one GPU shares that GPU's scratch: calls that may
 * overlap in time on one GPU (different streams, different host threads
 * without ordering) race and must not be made; calls in one stream's order
 * are safe.  Outputs, checks and errors are otherwise those of
 * lora_linear_bwd, whose kernels it runs. */
size_t lora_linear_bwd_noalloc_max_scratch(void);
lora_status lora_linear_bwd_noalloc(const void *dY, const void *X, const void *W, const void *A,
                                    const void *B, const float *S, const uint32_t *keep_bits,
                                    int64_t m, int64_t k, int64_t n, int32_t r, float alpha, float p,
                                    void *dX, void *dA, void *dB, hipStream_t stream);

/* ---- mixed-adapter batch (FusedMultiLoRA) ------------------------------- */

/* Segments: rows [seg_off[s], seg_off[s+1]) use adapter seg_adapter[s];
 * seg_off (int64, num_segments+1 entries) and seg_adapter (int32) are device
 * arrays; segments must be ordered, contiguous and cover [0, m); empty
 * segments are allowed.  r_max >= every adapter's r is the row stride of S.
 * Adapters are added to tiles of 128 rows with zeros in the rows of others: an
 * infinity or NaN in one adapter's A or B can make rows of its neighbours in
 * a tile NaN (finite adapters never touch each other's rows). */
size_t multi_lora_fwd_workspace_size(int64_t m, int64_t k, int64_t n, int32_t r_max,
                                     int32_t num_adapters, int32_t num_segments);

/* Forward for a mixed-adapter batch: Y (m x n), S (m x r_max; row i holds
 * its adapter's S, zero past that rank) and keep_bits (required). */
lora_status multi_lora_linear_fwd(const void *X, const void *W, const lora_adapter *adapters,
                                  int32_t num_adapters, const int64_t *seg_off,
                                  const int32_t *seg_adapter, int32_t num_segments,
                                  int64_t m, int64_t k, int64_t n, int32_t r_max,
                                  uint64_t seed, uint64_t offset,
                                  void *Y, float *S, uint32_t *keep_bits,
                                  void *workspace, size_t workspace_bytes, hipStream_t stream);

size_t multi_lora_bwd_workspace_size(int64_t m, int64_t k, int64_t n, int32_t r_max,
                                     int32_t num_adapters, int32_t num_segments);

/* Backward for a mixed-adapter batch: dX, and every adapter's dA and dB
 * (through the pointers in the adapter table; summed over all of that
 * adapter's rows; zero for adapters with no rows).  dX may be NULL: the input
 * gradient is then not computed. */
lora_status multi_lora_linear_bwd(const void *dY, const void *X, const void *W,
                                  const lora_adapter *adapters, int32_t num_adapters,
                                  const int64_t *seg_off, const int32_t *seg_adapter,
                                  int32_t num_segments, const float *S,
                                  const uint32_t *keep_bits, int64_t m, int64_t k, int64_t n,
                                  int32_t r_max, void *dX,
                                  void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Host: validate host copies of a segment table (0 if valid, else
 * LORA_ERR_INVALID_ARG with a message). */
lora_status multi_lora_check_segments(const int64_t *seg_off_host, const int32_t *seg_adapter_host,
                                      int32_t num_segments, int64_t m,
                                      const int32_t *adapter_r_host, int32_t num_adapters,
                                      int32_t r_max);

/* ---- mixed-adapter batching (host) ---------------------------------------
 * The step upstream of the mixed-adapter entry points: a scheduler packs the
 * samples of several adapters' global batches into microbatches of bounded
 * token count, and each microbatch's rows, grouped by adapter, become one
 * segment table (papers.chlience.com notes on LoRAFusion, section 4
 * "Multi-LoRA scheduler"; juhe.plus blog, section 4.2).  All arrays are host
 * memory owned by the caller; nothing is retained; no device work. */

/* Greedy packing of num_samples samples (lengths[i] tokens, 1 <= lengths[i]
 * <= capacity) into microbatches of at most `capacity` tokens: first-fit
 * decreasing -- samples longest first (equal lengths in index order), each
 * into the lowest-numbered microbatch with room, else into a new one (the
 * pages' greedy fallback of their MILP packer).  Writes mb_of_sample[i] (the
 * microbatch of sample i, numbered in opening order) and *num_microbatches.
 * LORA_ERR_INVALID_ARG for a length outside [1, capacity], capacity < 1,
 * num_samples < 0 or a NULL array. */
lora_status lora_pack_greedy(const int32_t *lengths, int32_t num_samples, int64_t capacity,
                             int32_t *mb_of_sample, int32_t *num_microbatches);

/* The segment table of microbatch `mb`: its samples ordered by adapter
 * (increasing id; one adapter's samples in increasing index), one segment per
 * adapter present.  Writes sample_order[0 .. *num_members) (sample indices in
 * row order; room for num_samples), seg_off[0 .. *num_segments] (token
 * offsets; room for num_adapters + 1; seg_off[*num_segments] is the
 * microbatch's row count m) and seg_adapter[0 .. *num_segments) (room for
 * num_adapters).  An empty microbatch gives zero segments and seg_off[0] = 0.
 * LORA_ERR_INVALID_ARG for an adapter id outside [0, num_adapters), a length
 * below 1 among the members, or a NULL array. */
lora_status lora_microbatch_segments(const int32_t *lengths, const int32_t *adapter_of_sample,
                                     const int32_t *mb_of_sample, int32_t num_samples,
                                     int32_t num_adapters, int32_t mb, int32_t *sample_order,
                                     int32_t *num_members, int64_t *seg_off,
                                     int32_t *seg_adapter, int32_t *num_segments);

/* Pipeline dependency check ("bubble lemma", same sections): with `stages`
 * pipeline stages, sample i sits in microbatch mb_of_sample[i] and belongs to
 * global batch batch_of_sample[i] of adapter adapter_of_sample[i].  For every
 * adapter and each of its global batches that has a later one with samples,
 * the earliest microbatch of that next batch must be at least the latest
 * microbatch of this batch plus stages - 1.  *violations = the number of
 * (adapter, batch) pairs that break it (0: the order is valid).
 * LORA_ERR_INVALID_ARG for stages < 1, an adapter id outside
 * [0, num_adapters), a negative index or a NULL array. */
lora_status lora_check_bubble_lemma(const int32_t *mb_of_sample, const int32_t *adapter_of_sample,
                                    const int32_t *batch_of_sample, int32_t num_samples,
                                    int32_t num_adapters, int32_t stages, int64_t *violations);

/* ---- DoRA norm -----------------------------------------------------------
 * DoRA rescales each output feature of the adapted weight by a learned
 * magnitude over its norm.  This computes that norm for every output feature
 * (a column here, since the layer is X W with W k x n):
 *   norm[j] = || W[:, j] + alpha * (A B)[:, j] ||_2
 * without storing the dense k x n product (page on the factored DoRA norm,
 * "core method": the norm of W + sBA per output feature, s the LoRA scale).
 * W (k x n), A (k x r) and B (r x n) are bf16 row-major device buffers,
 * 16-byte aligned; norm is n fp32 (4-byte aligned).  Sums are fp32 and
 * deterministic.  Requires 1 <= r <= 256, n % 8 == 0; the workspace holds
 * per-split partial sums (lora_dora_norm_workspace_size bytes, 16-byte
 * aligned).  LORA_ERR_UNSUPPORTED when A or B (with 32 spare rows) exceeds
 * 2 GiB. */
size_t lora_dora_norm_workspace_size(int64_t k, int64_t n, int32_t r);
lora_status lora_dora_norm(const void *W, const void *A, const void *B, int64_t k, int64_t n,
                           int32_t r, float alpha, float *norm, void *workspace,
                           size_t workspace_bytes, hipStream_t stream);

/* ---- frozen weights in 4 bits (MXFP4) ------------------------------------
 * The frozen W may be held in microscaled 4-bit floating point: e2m1 codes
 * (0, 1/2, 1, 3/2, 2, 3, 4, 6 and their negatives) in blocks of 32 along k
 * with one scale byte s per block, W'[i][j] = code * 2^(s - 127).  Every W'
 * is exactly a bf16.  The layers compute with W' in place of W, forward and
 * backward, and X, dY and the adapters stay bf16: the gradients are those of
 * the layer that the forward computed.
 *
 * Storage, N16 = ceil(n / 16) and KB = 4 ceil(k / 128):
 *   codes   [N16][KB][16][16] bytes: byte i of (c, b, j) holds W'[32b + 2i][16c + j]
 *           in its low nibble and W'[32b + 2i + 1][16c + j] in its high one
 *   scales  [N16][KB][16] bytes
 * both 16-byte aligned, lora_mxfp4_codes_size() and lora_mxfp4_scales_size()
 * bytes.  Padding columns and rows hold zero codes and scale bytes of 127, as
 * quantising writes them.
 *
 * lora_mxfp4_quantize: with a the block's largest magnitude, the scale is
 * 2^e, e = floor(log2 a) - 2, one more where a / 2^e >= 7, clamped to
 * [-125, 125]; each code is the nearest to w / 2^e (ties to the even code,
 * at most 6).  A block of zeros gets s = 127, and a block with an infinity or
 * a NaN s = 255: all its values then read as NaN.  Bytes 0, 1, 253 and 254
 * are not written by it but read as the powers of two they stand for (past
 * bf16's range as infinities). */
size_t lora_mxfp4_codes_size(int64_t k, int64_t n);
size_t lora_mxfp4_scales_size(int64_t k, int64_t n);
lora_status lora_mxfp4_quantize(const void *W, int64_t k, int64_t n, void *codes, void *scales,
                                hipStream_t stream);
/* W' as row-major k x n bf16 (exact). */
lora_status lora_mxfp4_dequantize(const void *codes, const void *scales, int64_t k, int64_t n, void *W,
                                  hipStream_t stream);

/* The frozen layer over W': Y = X W' and dX = dY W'^T.  m == 0 returns at
 * once. */
size_t lora_mxfp4_frozen_fwd_workspace_size(int64_t m, int64_t k, int64_t n);
lora_status lora_mxfp4_frozen_fwd(const void *X, const void *codes, const void *scales, int64_t m, int64_t k,
                                  int64_t n, void *Y, void *workspace, size_t workspace_bytes,
                                  hipStream_t stream);
size_t lora_mxfp4_frozen_bwd_workspace_size(int64_t m, int64_t k, int64_t n);
lora_status lora_mxfp4_frozen_bwd(const void *dY, const void *codes, const void *scales, int64_t m, int64_t k,
                                  int64_t n, void *dX, void *workspace, size_t workspace_bytes,
                                  hipStream_t stream);

/* lora_linear_fwd / lora_linear_bwd and multi_lora_linear_fwd / _bwd with W'
 * in place of W: the same arguments, outputs, checks and errors. */
size_t lora_mxfp4_linear_fwd_workspace_size(int64_t m, int64_t k, int64_t n, int32_t r);
lora_status lora_mxfp4_linear_fwd(const void *X, const void *codes, const void *scales, const void *A,
                                  const void *B, int64_t m, int64_t k, int64_t n, int32_t r, float alpha,
                                  float p, uint64_t seed, uint64_t offset, void *Y, float *S,
                                  uint32_t *keep_bits, void *workspace, size_t workspace_bytes,
                                  hipStream_t stream);
size_t lora_mxfp4_linear_bwd_workspace_size(int64_t m, int64_t k, int64_t n, int32_t r);
lora_status lora_mxfp4_linear_bwd(const void *dY, const void *X, const void *codes, const void *scales,
                                  const void *A, const void *B, const float *S, const uint32_t *keep_bits,
                                  int64_t m, int64_t k, int64_t n, int32_t r, float alpha, float p, void *dX,
                                  void *dA, void *dB, void *workspace, size_t workspace_bytes,
                                  hipStream_t stream);
size_t multi_lora_mxfp4_fwd_workspace_size(int64_t m, int64_t k, int64_t n, int32_t r_max,
                                           int32_t num_adapters, int32_t num_segments);
lora_status multi_lora_mxfp4_linear_fwd(const void *X, const void *codes, const void *scales,
                                        const lora_adapter *adapters, int32_t num_adapters,
                                        const int64_t *seg_off, const int32_t *seg_adapter,
                                        int32_t num_segments, int64_t m, int64_t k, int64_t n, int32_t r_max,
                                        uint64_t seed, uint64_t offset, void *Y, float *S,
                                        uint32_t *keep_bits, void *workspace, size_t workspace_bytes,
                                        hipStream_t stream);
size_t multi_lora_mxfp4_bwd_workspace_size(int64_t m, int64_t k, int64_t n, int32_t r_max,
                                           int32_t num_adapters, int32_t num_segments);
lora_status multi_lora_mxfp4_linear_bwd(const void *dY, const void *X, const void *codes, const void *scales,
                                        const lora_adapter *adapters, int32_t num_adapters,
                                        const int64_t *seg_off, const int32_t *seg_adapter,
                                        int32_t num_segments, const float *S, const uint32_t *keep_bits,
                                        int64_t m, int64_t k, int64_t n, int32_t r_max, void *dX,
                                        void *workspace, size_t workspace_bytes, hipStream_t stream);

/* ---- frozen weights of 4-bit integers in groups of rows --------------------
 * The frozen W may also be held as 4-bit integers q with one scale s and one
 * zero z for `group` rows of a column, W'[i][j] = s (q - z), which is how
 * integer-quantised checkpoints hold it.  group is 32, 64 or a multiple of
 * 128 (k or more rows: one scale a column).
 *
 * Storage, N16 = ceil(n / 16) and K128 = ceil(k / 128):
 *   codes   [N16][K128][4][16][16] bytes: word d (little-endian) of the 16
 *           bytes of (c, t, g, j) holds rows i .. i+7, i = 128t + 32d + 8g, of
 *           column 16c + j; rows i, i+2, i+4, i+6 in its low four nibbles
 *           from the lowest up, i+1, i+3, i+5, i+7 in its high four
 *   scales  [N16][G][16] words: the bits of s as a float with its last 8 bits
 *           zero, and z (0 .. 255) in those 8, of column 16c + j;
 *           G = 128 K128 / group for groups of 32 or 64, else ceil(k / group)
 * both 16-byte aligned, lora_int4_codes_size() and lora_int4_scales_size()
 * bytes.  s has 16 significant bits: a bf16's or an fp16's exactly.  Padding
 * columns and rows hold code 0, padding columns and groups the word 0.
 *
 * lora_int4_quantize makes both from a bf16 W, to the nearest code (ties of
 * w / s to even, then clamped to 0 .. 15):
 *   symmetric = 0: lo and hi the group's smallest and largest value and 0,
 *                  s = (hi - lo) / 15, z = -lo / s to the nearest integer
 *   symmetric = 1: s = max |w| / 7, z = 8
 * s rounded to 16 significant bits and at least 2^-120; a group of zeros has
 * s = 1, one with an infinity or a NaN has s = NaN: all its values then are.
 *
 * lora_int4_pack makes both from a checkpoint's: Q (k x n bytes, the code in
 * the low four bits), group_scales (ceil(k / group) x n of scale_type 0: fp32,
 * rounded to 16 significant bits, 1: bf16, 2: fp16; an infinity, given or
 * rounded to, reads as NaN) and zeros (ceil(k / group) x n bytes; NULL: every
 * zero is 8); Q and group_scales 4-byte aligned. */
size_t lora_int4_codes_size(int64_t k, int64_t n);
size_t lora_int4_scales_size(int64_t k, int64_t n, int64_t group);
lora_status lora_int4_quantize(const void *W, int64_t k, int64_t n, int64_t group, int32_t symmetric, void *codes,
                               void *scales, hipStream_t stream);
lora_status lora_int4_pack(const void *Q, const void *group_scales, int32_t scale_type, const void *zeros, int64_t k,
                           int64_t n, int64_t group, void *codes, void *scales, hipStream_t stream);
/* W' as row-major k x n bf16, each value rounded to the nearest. */
lora_status lora_int4_dequantize(const void *codes, const void *scales, int64_t k, int64_t n, int64_t group, void *W,
                                 hipStream_t stream);

/* The frozen layer and the LoRA layers over W': as lora_frozen_fwd / _bwd,
 * lora_linear_fwd / _bwd and multi_lora_linear_fwd / _bwd, with the same
 * arguments, outputs, checks and errors.
 *
 * A forward multiplies W' as it is where it reads the packed weight, group by
 * group in fp32: always for up to 64 rows with k <= 2^20 and n <= 2^24, and for
 * more rows where that is faster than expanding W' into the workspace.  A
 * larger weight is expanded at any row count.  An expanded W', and W' in every
 * backward, has each of its values rounded to bf16.  Equal sizes take equal
 * ways.  In a forward from the packed weight a row's products are sums of
 * x (16 + q) less (16 + z) times the sum of x: a row of X with an infinity
 * gives NaN, as does one whose sum of 271 |x| over a group is past fp32's
 * range. */
size_t lora_int4_frozen_fwd_workspace_size(int64_t m, int64_t k, int64_t n, int64_t group);
lora_status lora_int4_frozen_fwd(const void *X, const void *codes, const void *scales, int64_t group, int64_t m,
                                 int64_t k, int64_t n, void *Y, void *workspace, size_t workspace_bytes,
                                 hipStream_t stream);
size_t lora_int4_frozen_bwd_workspace_size(int64_t m, int64_t k, int64_t n, int64_t group);
lora_status lora_int4_frozen_bwd(const void *dY, const void *codes, const void *scales, int64_t group, int64_t m,
                                 int64_t k, int64_t n, void *dX, void *workspace, size_t workspace_bytes,
                                 hipStream_t stream);
size_t lora_int4_linear_fwd_workspace_size(int64_t m, int64_t k, int64_t n, int64_t group, int32_t r);
lora_status lora_int4_linear_fwd(const void *X, const void *codes, const void *scales, int64_t group, const void *A,
                                 const void *B, int64_t m, int64_t k, int64_t n, int32_t r, float alpha, float p,
                                 uint64_t seed, uint64_t offset, void *Y, float *S, uint32_t *keep_bits,
                                 void *workspace, size_t workspace_bytes, hipStream_t stream);
size_t lora_int4_linear_bwd_workspace_size(int64_t m, int64_t k, int64_t n, int64_t group, int32_t r);
lora_status lora_int4_linear_bwd(const void *dY, const void *X, const void *codes, const void *scales, int64_t group,
                                 const void *A, const void *B, const float *S, const uint32_t *keep_bits, int64_t m,
                                 int64_t k, int64_t n, int32_t r, float alpha, float p, void *dX, void *dA, void *dB,
                                 void *workspace, size_t workspace_bytes, hipStream_t stream);
size_t multi_lora_int4_fwd_workspace_size(int64_t m, int64_t k, int64_t n, int64_t group, int32_t r_max,
                                          int32_t num_adapters, int32_t num_segments);
lora_status multi_lora_int4_linear_fwd(const void *X, const void *codes, const void *scales, int64_t group,
                                       const lora_adapter *adapters, int32_t num_adapters, const int64_t *seg_off,
                                       const int32_t *seg_adapter, int32_t num_segments, int64_t m, int64_t k,
                                       int64_t n, int32_t r_max, uint64_t seed, uint64_t offset, void *Y, float *S,
                                       uint32_t *keep_bits, void *workspace, size_t workspace_bytes,
                                       hipStream_t stream);
size_t multi_lora_int4_bwd_workspace_size(int64_t m, int64_t k, int64_t n, int64_t group, int32_t r_max,
                                          int32_t num_adapters, int32_t num_segments);
lora_status multi_lora_int4_linear_bwd(const void *dY, const void *X, const void *codes, const void *scales,
                                       int64_t group, const lora_adapter *adapters, int32_t num_adapters,
                                       const int64_t *seg_off, const int32_t *seg_adapter, int32_t num_segments,
                                       const float *S, const uint32_t *keep_bits, int64_t m, int64_t k, int64_t n,
                                       int32_t r_max, void *dX, void *workspace, size_t workspace_bytes,
                                       hipStream_t stream);

/* ---- the layer's input saved in 8 bits (MXINT8) -----------------------------
 * X is all that the backward keeps of a layer that grows with tokens times
 * width, and it is read for dA alone.  It may be saved as 8-bit integers in
 * blocks of 32 along each row with one power-of-two scale byte s each,
 * X'[i][32b + j] = c 2^(s - 127), 0.52 of its bf16 bytes.  Every X' is exactly
 * a bf16.
 *
 * Storage, KB = 4 ceil(k / 128): codes [m][KB][32] int8 (16-byte aligned) and
 * scales [m][KB] bytes (4-byte aligned).  Padding holds codes 0, scales 127.
 *
 * lora_mxint8_quantize: with a the block's largest magnitude, the scale is
 * 2^e, e = floor(log2 a) - 6 clamped to [-120, 121], and each code the nearest
 * to x / 2^e (ties to even): |x - x'| <= 2^(e-1).  A block of zeros gets
 * s = 127, and a block with an infinity or a NaN s = 255: all its values then
 * read as NaN.  Other bytes that are not written by it read as the powers of
 * two they stand for. */
size_t lora_mxint8_codes_size(int64_t m, int64_t k);
size_t lora_mxint8_scales_size(int64_t m, int64_t k);
lora_status lora_mxint8_quantize(const void *X, int64_t m, int64_t k, void *codes, void *scales, hipStream_t stream);
/* X' as row-major m x k bf16 (exact). */
lora_status lora_mxint8_dequantize(const void *codes, const void *scales, int64_t m, int64_t k, void *X,
                                   hipStream_t stream);

/* lora_linear_bwd and multi_lora_linear_bwd with X' in place of X (S and
 * keep_bits are the forward's, which ran on X): dA = s (keep (.) X')^T dS, and
 * dX and dB as before.  The weight is W (kind LORA_WEIGHT_BF16; W_scales and
 * group are not read), the codes and scales of an MXFP4 weight (group is not
 * read) or those of 4-bit integers.  Other arguments, outputs, checks and
 * errors as there; with one adapter and a dX, A's 2 GiB are counted with r
 * rounded up to 8. */
typedef enum { LORA_WEIGHT_BF16 = 0, LORA_WEIGHT_MXFP4 = 1, LORA_WEIGHT_INT4 = 2 } lora_weight_kind;
size_t lora_mxint8_linear_bwd_workspace_size(int32_t kind, int64_t group, int64_t m, int64_t k, int64_t n, int32_t r);
lora_status lora_mxint8_linear_bwd(const void *dY, const void *x_codes, const void *x_scales, int32_t kind,
                                   const void *W, const void *W_scales, int64_t group, const void *A, const void *B,
                                   const float *S, const uint32_t *keep_bits, int64_t m, int64_t k, int64_t n,
                                   int32_t r, float alpha, float p, void *dX, void *dA, void *dB, void *workspace,
                                   size_t workspace_bytes, hipStream_t stream);
size_t multi_lora_mxint8_bwd_workspace_size(int32_t kind, int64_t group, int64_t m, int64_t k, int64_t n,
                                            int32_t r_max, int32_t num_adapters, int32_t num_segments);
lora_status multi_lora_mxint8_linear_bwd(const void *dY, const void *x_codes, const void *x_scales, int32_t kind,
                                         const void *W, const void *W_scales, int64_t group,
                                         const lora_adapter *adapters, int32_t num_adapters, const int64_t *seg_off,
                                         const int32_t *seg_adapter, int32_t num_segments, const float *S,
                                         const uint32_t *keep_bits, int64_t m, int64_t k, int64_t n, int32_t r_max,
                                         void *dX, void *workspace, size_t workspace_bytes, hipStream_t stream);

/* ---- optimizer ------------------------------------------------------------
 * One AdamW step over many tensors (the adapters' A and B of a model):
 *   m = beta1 m + (1 - beta1) g       v = beta2 v + (1 - beta2) g^2
 *   w = w - (lr weight_decay w + lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps))
 * in fp32 (each constant, 1 - beta and lr weight_decay among them, rounded from its
 * double; the two terms are added before w takes them, in one rounding), everything
 * updated in place.
 *
 * Types: param is fp32, or bf16 (param_bf16 = 1) with or without an fp32
 * master copy; with one the master is updated and param becomes its nearest
 * bf16, without one w is read from param and rounded to it.  grad is fp32 or
 * bf16 (grad_bf16 = 1).  state_bits = 32: m and v are n floats.
 * state_bits = 8: m and v are n e4m3 bytes (OCP FP8), codes of m and of
 * sqrt(v), and m_scale and v_scale ceil(n / 256) floats: value = code * scale
 * of its block of 256.  A new moment x of a block with largest magnitude a
 * becomes scale = a / 448 and a code drawn between the two neighbours of
 * x / scale so that its mean is x / scale (a positive root keeps at least the
 * smallest code, so the division stays bounded; a below 2^-100 gives zeros, and
 * v below the smallest normal float, 2^-126, has the root zero).
 * The draw of value i is word (offset + i) % 4 of Philox4x32-10 at counter
 * (offset + i) / 4 under key seed + t * 0x9E3779B97F4A7C15 (mod 2^64), its low
 * half for m and its high half for v.  offset is a multiple of 8; tensors
 * with disjoint ranges [offset, offset + n) draw independently.
 *
 * An infinite or NaN gradient makes its own w and moments NaN (or infinite)
 * and nothing else.  eps is 0 or at least 2^-126, the smallest normal float; with
 * eps = 0 a value whose gradients were all zero becomes NaN, as 0 / 0 does.
 *
 * t = step (>= 1) or, where step_dev is not NULL, the int64 it points to on
 * the device, read when the kernels run (a captured call then follows the
 * caller's counter; with `step` a replay repeats the captured t).
 *
 * `tensors` is a host array, read during the call only.  Records with n = 0
 * are skipped.  Either every record has a master copy or none.  No two
 * records may share memory that the call writes. */
typedef struct {
    void *param;
    const void *grad;
    float *master;
    void *m;
    void *v;
    float *m_scale;
    float *v_scale;
    int64_t n;
    uint64_t offset;
} lora_adamw_tensor;

lora_status lora_adamw_step(const lora_adamw_tensor *tensors, int32_t count, int32_t param_bf16,
                            int32_t grad_bf16, int32_t state_bits, double lr, double beta1,
                            double beta2, double eps, double weight_decay, int64_t step,
                            const int64_t *step_dev, uint64_t seed, hipStream_t stream);

/* ---- pieces exposed for testing and as the frozen-layer baseline -------- */

/* The dropout mask alone (same bits the forward stores). */
lora_status lora_dropout_mask(uint64_t seed, uint64_t offset, int64_t m, int64_t k, float p,
                              uint32_t *keep_bits, hipStream_t stream);

/* Frozen linear layer, forward Y = X W and backward dX = dY W^T, on the same
 * MFMA GEMM as the LoRA path (the frozen layer the pages compare against:
 * papers.chlience.com notes, "Result 1: LoRA overhead profiling"). */
lora_status lora_frozen_fwd(const void *X, const void *W, int64_t m, int64_t k, int64_t n,
                            void *Y, hipStream_t stream);
lora_status lora_frozen_bwd(const void *dY, const void *W, int64_t m, int64_t k, int64_t n,
                            void *dX, hipStream_t stream);

/* ---- kernel timing (tracing) --------------------------------------------
 * When enabled, every kernel the library launches is bracketed by a pair of
 * HIP events recorded on the launch stream.  lora_profiling_query()
 * synchronises those events and returns, for kernels whose name contains
 * `name_substring`, the number of launches and their summed duration in
 * milliseconds since the last reset.  Event pairs come from a pool created by
 * lora_profiling_enable(1) (capacity events per kernel launch slot); launches
 * beyond the capacity are not timed.  The products over an MXFP4 weight carry
 * their tile ("mxfp4_gemm 64x128", "mxfp4_gemm_t 128x256"). */
lora_status lora_profiling_enable(int32_t enable, int32_t capacity);
lora_status lora_profiling_reset(void);
lora_status lora_profiling_query(const char *name_substring, int64_t *launches, double *total_ms);

/* ---- status ------------------------------------------------------------ */
const char *lora_status_string(lora_status s);
const char *lora_last_error_message(void);

#ifdef __cplusplus
}
#endif

#endif /* LORA_FUSED_H */
