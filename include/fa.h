/*
 * fa.h -- C ABI of the exact tiled attention library for NVIDIA GB300 (sm_103a).
 *
 * Two operations, as the source pages define them, and for the second an 8-bit paged KV cache
 * (fa_kv_append_paged_fp8, fa_kv_read_paged_fp8, fa_decode_splitkv_paged_fp8) and the operators of
 * a serving loop over the 16-bit one (fa_kv_append_paged_rope, fa_decode_splitkv_paged_tree,
 * fa_decode_splitkv_paged_window, with fa_fwd_sinks and fa_fwd_varlen_sinks for its prompts):
 *
 *  fa_fwd             exact attention forward, O = softmax(scale * Q K^T [+ causal mask]) V,
 *                     plus the per-row log-sum-exp.  Page "flash-attention-v100", section
 *                     "How to use FlashAttention" (flash_attn_func: tensors
 *                     (batch, seqlen, nheads, headdim), grouped-query heads, default scale
 *                     1/sqrt(headdim)); section "Changelog", "2.1: Change behavior of causal
 *                     flag" (bottom-right aligned mask, all-masked rows give zero output);
 *                     page "ampere_flash_attention_from_scratch" (the FlashAttention-2 forward
 *                     that tiles Q row blocks over thread blocks and streams K/V tiles).
 *
 *  fa_decode_splitkv  single-token decode over a KV cache with per-sequence lengths, the KV
 *                     range cut into pieces processed by different thread blocks, each
 *                     writing a partial output and its log-sum-exp, then merged by a
 *                     separate kernel.  Page "flash-attention-v100", "Changelog",
 *                     "2.2: Optimize for inference" and flash_attn_with_kvcache
 *                     (cache_seqlens); page "flash attention-2 github" (Flash-Decoding,
 *                     steps 1-3).
 *
 * Conventions for every entry point:
 *  - Tensors are contiguous, row-major, 16-bit (bf16 or fp16 as `dtype` says):
 *    Q [B, Sq, Hq, D], K and V [B, Sk, Hkv, D], O [B, Sq, Hq, D]; LSE is fp32 [B, Hq, Sq].
 *    Hq must be a multiple of Hkv; Q head h reads K/V head h / (Hq / Hkv).
 *  - All pointers are device memory owned by the caller and must be 16-byte aligned.
 *    The library allocates nothing on these paths; the decode workspace is sized by
 *    fa_decode_workspace_bytes() and passed in.
 *  - Work is enqueued on `stream` and runs asynchronously; no entry point synchronises.
 *    Arguments are validated before anything is enqueued: a bad argument returns an error
 *    and enqueues nothing.  FA_ERR_CUDA reports a launch failure (cudaGetLastError).
 *  - Kernel-side waits are bounded: a wait that exceeds its limit makes the kernel unwind
 *    and records FA_ERR_TIMEOUT, read back with fa_last_device_status().
 *  - No C++ exception crosses this interface.
 */
#ifndef FA_H_
#define FA_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define FA_API __attribute__((visibility("default")))
#else
#define FA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st *fa_stream_t;

typedef enum {
    FA_OK = 0,
    FA_ERR_INVALID_ARG = 1, /* null/misaligned pointer, non-positive size, Hq % Hkv != 0 */
    FA_ERR_UNSUPPORTED = 2, /* head dim not in {64, 96, 128, 256}, unknown dtype */
    FA_ERR_WORKSPACE = 3,   /* decode workspace missing or smaller than required */
    FA_ERR_CUDA = 4,        /* a CUDA runtime / driver call failed */
    FA_ERR_TIMEOUT = 5      /* a kernel gave up on a bounded wait (see fa_last_device_status) */
} fa_status;

typedef enum { FA_BF16 = 0, FA_FP16 = 1 } fa_dtype;

/*
 * Exact attention forward (FlashAttention-2 style: Q row blocks in parallel, K/V tiles
 * streamed, online softmax, the Sq x Sk score matrix never stored).
 *   q     [B, Sq, Hq, D]    k, v  [B, Sk, Hkv, D]    o  [B, Sq, Hq, D]  (dtype)
 *   lse   [B, Hq, Sq] fp32, natural log of sum_j exp(scale * q_i . k_j) over the visible
 *         keys; -inf for a row with no visible key (whose output row is 0).  May be NULL.
 *   scale softmax scale (the pages' default is 1/sqrt(D); the caller passes it).
 *   causal nonzero: key j is visible to query i iff j <= i + Sk - Sq.
 * Sizes: B, Sq, Sk, Hq, Hkv >= 1; D in {64, 96, 128, 256}; Hq % Hkv == 0.
 * Accumulation is fp32; P is rounded to the input dtype before the P.V product; O is
 * rounded once (round-to-nearest-even).  Deterministic: the same inputs give the same bits.
 */
FA_API fa_status fa_fwd(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Sq,
                 int Sk, int Hq, int Hkv, int D, float scale, int causal, fa_dtype dtype,
                 fa_stream_t stream);

/*
 * fa_fwd restricted to a sliding window (local attention; page "flash-attention-v100",
 * flash_attn_func window_size, and "Changelog", "2.3: Local (i.e., sliding window)
 * attention"): query i attends only to keys j with
 *     i + Sk - Sq - window_left <= j <= i + Sk - Sq + window_right,
 * where -1 leaves that side unbounded, as any side past every key does; with causal != 0 the
 * right bound is additionally j <= i + Sk - Sq.  K/V blocks outside every row's window are
 * skipped, not masked.  A row whose window holds no key gets O = 0 and LSE = -inf.
 * window_left/right >= -1, else FA_ERR_INVALID_ARG; everything else as fa_fwd (which equals
 * window (-1, -1)).
 */
FA_API fa_status fa_fwd_window(const void *q, const void *k, const void *v, void *o, float *lse,
                               int B, int Sq, int Sk, int Hq, int Hkv, int D, float scale,
                               int causal, int window_left, int window_right, fa_dtype dtype,
                               fa_stream_t stream);

/*
 * Variable-length batch (page "flash-attention-v100", "Changelog", "2.0",
 * flash_attn_varlen_func): the B sequences are packed along the rows.
 *   q, o          [total_q, Hq, D]     k, v  [total_k, Hkv, D]      (dtype)
 *   cu_seqlens_q  device int32 [B + 1]: sequence b owns query rows
 *                 [cu_seqlens_q[b], cu_seqlens_q[b + 1]); cu_seqlens_k likewise for keys;
 *                 both non-decreasing, from 0, ending at most at total_q / total_k.
 *   lse           [Hq, total_q] fp32 (may be NULL).
 * Within a sequence everything is as fa_fwd_window: the causal mask is aligned to that
 * sequence's bottom-right corner.  A sequence with no keys gets O = 0 and LSE = -inf.
 * B <= 1024.  The offsets are read on the device; rows they place outside [0, total_q)
 * are not written, and keys outside [0, total_k) read as zero.
 */
FA_API fa_status fa_fwd_varlen(const void *q, const void *k, const void *v, void *o, float *lse,
                               const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int B,
                               int total_q, int total_k, int Hq, int Hkv, int D, float scale,
                               int causal, int window_left, int window_right, fa_dtype dtype,
                               fa_stream_t stream);

/*
 * fa_fwd_window and fa_fwd_varlen with sinks: the first `sinks` keys of a sequence stay visible
 * left of the window.  Query i sees the keys j with
 *     j <= i + Sk - Sq + window_right  (the right side as without sinks), and
 *     j >= i + Sk - Sq - window_left  or  j < sinks.
 * Blocks of keys between the sinks and every row's window are skipped.  What a row does not see is
 * not used for it, NaN and infinities included; where a V that is not finite meets a row's block, the
 * tiles around it are gone through a second time.  o must not overlap q, k or v.  sinks >= 0, and
 * scale > 0 if there are any, else FA_ERR_INVALID_ARG.  Where the sinks do not matter (sinks == 0, or
 * window_left == -1 or at least the keys) the call is fa_fwd_window (fa_fwd_varlen), where a hidden V
 * that is not finite can give NaN; everything else as there.
 */
FA_API fa_status fa_fwd_sinks(const void *q, const void *k, const void *v, void *o, float *lse,
                              int B, int Sq, int Sk, int Hq, int Hkv, int D, float scale,
                              int causal, int window_left, int window_right, int sinks,
                              fa_dtype dtype, fa_stream_t stream);

FA_API fa_status fa_fwd_varlen_sinks(const void *q, const void *k, const void *v, void *o,
                                     float *lse, const int32_t *cu_seqlens_q,
                                     const int32_t *cu_seqlens_k, int B, int total_q, int total_k,
                                     int Hq, int Hkv, int D, float scale, int causal,
                                     int window_left, int window_right, int sinks, fa_dtype dtype,
                                     fa_stream_t stream);

/*
 * Bytes of decode workspace fa_decode_splitkv needs for these sizes and `num_splits`
 * (the partial outputs [B, Hq, num_splits, D] fp32 and their log-sum-exps
 * [B, Hq, num_splits] fp32, each region 256-byte aligned).  0 for invalid sizes.
 * Host-only; needs no GPU.
 */
FA_API size_t fa_decode_workspace_bytes(int B, int Hq, int D, int num_splits);

/*
 * The split count fa_decode_splitkv uses when given num_splits <= 0: about eight partials
 * per SM over the B * Hkv (sequence, kv head) pairs, and no more than one per 256 keys of
 * max_kv_len.  It bounds how finely a pair may be cut (see num_splits below).  max_kv_len
 * is an upper bound on the KV lengths (the cache capacity Smax will do).  num_sms <= 0
 * queries the current device.  Returns >= 1, or -1 on an invalid argument or when no
 * device can be queried.
 */
FA_API int fa_decode_default_splits(int B, int Hkv, int max_kv_len, int num_sms);

/*
 * Split-KV decode for one query token per sequence.
 *   q        [B, 1, Hq, D]   k_cache, v_cache [B, Smax, Hkv, D]   (dtype)
 *   kv_lens  device int32 [B], 0 <= kv_lens[b] <= Smax: sequence b attends to cache
 *            positions [0, kv_lens[b]).  kv_lens[b] == 0 gives o = 0, lse = -inf.
 *   o        [B, 1, Hq, D] (dtype)      lse [B, Hq] fp32 (may be NULL)
 *   num_splits  the most pieces any (sequence, kv head) pair is cut into (<= 0: the
 *            default above).  The keys of all pairs, in 128-key tiles, are laid end to end
 *            in (b, kv head) order and cut into one equal range of W tiles per SM, W at
 *            least ceil(T / (num_splits - 1)) for the longest pair's T tiles (with
 *            num_splits == 1 no pair is cut).  Each piece of a pair writes a partial
 *            output and log-sum-exp, and a second kernel merges each pair's pieces.
 *            The kv heads are laid out in groups of g adjacent heads, g the largest of
 *            8, 4 and 2 that divides Hkv (else 1): a group is one entry, whose tiles count
 *            once, and the ranges go one per g SMs (the SM count rounded down to a
 *            multiple of g), one SM per head, so that the heads of a group get the same
 *            pieces and read the rows that sit side by side in the cache together.
 *   workspace   device memory of at least fa_decode_workspace_bytes(B, Hq, D, num_splits)
 *            bytes (after the default is applied); its contents need no initialisation.
 * Sizes: B, Hq, Hkv, Smax >= 1; B <= 1024; D in {64, 96, 128, 256}; Hq % Hkv == 0;
 * Hq / Hkv <= 16.
 * The result does not depend on num_splits beyond fp32 rounding.  Values of kv_lens
 * outside [0, Smax] are the caller's error and are clamped on the device.
 */
FA_API fa_status fa_decode_splitkv(const void *q, const void *k_cache, const void *v_cache,
                            const int32_t *kv_lens, void *o, float *lse, int B, int Hq, int Hkv,
                            int D, int Smax, float scale, int num_splits, void *workspace,
                            size_t workspace_bytes, fa_dtype dtype, fa_stream_t stream);

/*
 * Split-KV decode with Sq >= 1 query tokens per sequence (speculative or chunked decoding;
 * page "flash-attention-v100", flash_attn_with_kvcache with seqlen_q > 1 and the causal
 * flag of "Changelog", "2.1").
 *   q, o      [B, Sq, Hq, D] (dtype)     lse [B, Hq, Sq] fp32 (may be NULL)
 *   causal    nonzero: token s of sequence b sees cache keys j <= kv_lens[b] - Sq + s
 *             (the bottom-right aligned mask); zero: every token sees [0, kv_lens[b]).
 * (Hq / Hkv) * Sq <= 16.  The workspace is fa_decode_workspace_bytes(B * Sq, Hq, D,
 * num_splits).  A token that sees no key gets O = 0 and LSE = -inf.  Everything else as
 * fa_decode_splitkv, which is the Sq = 1 case.
 */
FA_API fa_status fa_decode_splitkv_multi(const void *q, const void *k_cache, const void *v_cache,
                                         const int32_t *kv_lens, void *o, float *lse, int B,
                                         int Sq, int Hq, int Hkv, int D, int Smax, float scale,
                                         int causal, int num_splits, void *workspace,
                                         size_t workspace_bytes, fa_dtype dtype,
                                         fa_stream_t stream);

/*
 * fa_decode_splitkv over a paged KV cache (page "flash-attention-v100",
 * flash_attn_with_kvcache with block_table; "Changelog", "2.5: Paged KV cache").
 *   k_pages, v_pages   [num_pages, page_size, Hkv, D] (dtype): a pool of pages
 *   block_table        device int32 [B, max_pages_per_seq]: key r of sequence b is row
 *                      r % page_size of page block_table[b][r / page_size]
 *   kv_lens            device int32 [B], 0 <= kv_lens[b] <= page_size * max_pages_per_seq
 * page_size must be a multiple of 128 (the pages ask for multiples of 256, which are
 * accepted).  Table entries outside [0, num_pages) for pages a sequence uses are the
 * caller's error: those keys read as zeros, never outside the pool.  Everything else,
 * including the workspace (fa_decode_workspace_bytes(B, Hq, D, num_splits)) and the
 * split into pieces, is as fa_decode_splitkv with Smax = page_size * max_pages_per_seq.
 */
FA_API fa_status fa_decode_splitkv_paged(const void *q, const void *k_pages, const void *v_pages,
                                         const int32_t *block_table, const int32_t *kv_lens,
                                         void *o, float *lse, int B, int Hq, int Hkv, int D,
                                         int num_pages, int page_size, int max_pages_per_seq,
                                         float scale, int num_splits, void *workspace,
                                         size_t workspace_bytes, fa_dtype dtype,
                                         fa_stream_t stream);

/*
 * Split-KV decode for callers that cannot allocate device memory -- for example a plugin
 * running inside a host runtime that owns every device allocation, or a latency-critical
 * serving loop that must never call cudaMalloc (which may synchronise the device).  The
 * source pages have no counterpart to this entry point; it exists for those callers.
 *
 * Same arguments and results as fa_decode_splitkv, minus the workspace: the partial
 * results go to a fixed scratch array of FA_DECODE_NOALLOC_SCRATCH_BYTES that lives in
 * the library's device image (every GPU that loads the library holds it until the process
 * exits).  The call allocates nothing and calls no allocating routine.
 *  - Limit: sizes whose workspace, fa_decode_workspace_bytes(B, Hq, D, num_splits) after
 *    the default split count is applied, exceeds FA_DECODE_NOALLOC_SCRATCH_BYTES are
 *    rejected with FA_ERR_WORKSPACE before anything is enqueued.
 *  - Set-up: the first call on each device (with that device current) looks up the
 *    array's device address once and keeps it; later calls reuse it.
 *  - Sharing: every call on a device uses the same array and leaves its contents behind.
 *    Nothing in it needs to start at zero (each call writes every partial it reads), but
 *    calls whose kernels overlap on the GPU (e.g. on two streams at once) race on it.
 */
#define FA_DECODE_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)

FA_API fa_status fa_decode_splitkv_noalloc(const void *q, const void *k_cache,
                                           const void *v_cache, const int32_t *kv_lens, void *o,
                                           float *lse, int B, int Hq, int Hkv, int D, int Smax,
                                           float scale, int num_splits, fa_dtype dtype,
                                           fa_stream_t stream);

/*
 * 8-bit paged KV cache.  The pages' changelog quantises nothing; these three entry points
 * are this library's own: a paged cache at half the bytes of the 16-bit one, written,
 * attended over and read back.
 *
 * A row is one token's D values of one kv head, held as e4m3 codes (4 significant bits)
 * with one power-of-two scale:
 *   k_pages, v_pages    [num_pages, Hkv, page_size, D]  e4m3 codes
 *   k_scales, v_scales  [num_pages, Hkv, page_size]     bytes s; the scale is 2^(s - 127)
 * and stands for code * 2^(s - 127), 0 <= s <= 254 (the append writes 247 at most; what a key with
 * s = 255 that a call uses gives is not specified).  The head comes before the slot, other than in the
 * 16-bit pools, so that what one head reads of a page is one run of memory.
 *   block_table         device int32 [B, max_pages_per_seq]: key r of sequence b is slot
 *                       r % page_size of page block_table[b][r / page_size]
 * page_size is a multiple of 16; D in {64, 96, 128, 256}; B <= 1024;
 * page_size * max_pages_per_seq <= 2^31 - 4096; num_pages * Hkv * page_size / 16 < 2^31; the
 * pools and scales are 16-byte aligned.  Table
 * entries outside [0, num_pages) that a call meets are the caller's error: nothing is read
 * or written outside the pool (what happens instead is said at each call).  Outputs and the
 * workspace must not overlap the inputs.  A contiguous
 * cache of Smax keys per sequence (a multiple of 16) is the pool with page_size = Smax and
 * block_table[b][0] = b.  `dtype` is the type of the 16-bit side; rows may be written in one and read or
 * attended over in the other.
 *
 * fa_kv_append_paged_fp8 quantises new rows as it writes them.
 *   k_new, v_new    token t, kv head h at element t * k_stride (v_stride) + h * D, so the
 *                   rows may lie inside a fused projection's output; strides in elements,
 *                   multiples of 8, at least Hkv * D; 16-byte aligned
 *   cu_seqlens_new  device int32 [B + 1]: sequence b's new tokens are packed rows
 *                   [cu_seqlens_new[b], cu_seqlens_new[b + 1]), non-decreasing, ending at
 *                   most at total_new; rows behind the last are not written.  NULL: every
 *                   sequence has total_new / B new tokens (B must divide total_new)
 *   kv_lens         device int32 [B]: sequence b's keys INCLUDING the new ones: its new
 *                   tokens become its last keys, kv_lens[b] - n .. kv_lens[b] - 1 (what a
 *                   decode with the same kv_lens then sees)
 * A row's scale is the least 2^e, e >= -127, with max |x| <= 448 * 2^e (448: e4m3's largest
 * value), and its codes are x / 2^e rounded to nearest even: a value is off by at most
 * 2^-4 of itself, or 2^(e - 10) where that is more.  A value that is not finite takes no
 * part in the scale and becomes NaN.  total_new == 0 writes nothing (k_new and v_new may
 * then be NULL).  Rows whose key is outside [0, page_size * max_pages_per_seq) or whose
 * page is outside the pool are dropped.  Two tokens that name the same slot of a page in
 * one call are the caller's error; the slot then holds one of them or a mixture.
 */
FA_API fa_status fa_kv_append_paged_fp8(const void *k_new, const void *v_new, int64_t k_stride,
                                        int64_t v_stride, const int32_t *cu_seqlens_new,
                                        const int32_t *block_table, const int32_t *kv_lens,
                                        void *k_pages, void *v_pages, uint8_t *k_scales,
                                        uint8_t *v_scales, int B, int total_new, int Hkv, int D,
                                        int num_pages, int page_size, int max_pages_per_seq,
                                        fa_dtype dtype, fa_stream_t stream);

/*
 * Reads rows of the 8-bit paged cache back as `dtype`, packed along the sequences: the K
 * and V of an fa_fwd_varlen over an already cached prefix.
 *   cu_seqlens  device int32 [B + 1]: packed rows [cu_seqlens[b], cu_seqlens[b + 1]) of k
 *               and v receive sequence b's keys kv_starts[b], kv_starts[b] + 1, ...
 *   kv_starts   device int32 [B]; NULL: 0 for every sequence
 *   k, v        [total, Hkv, D] (dtype)
 * Rows that no sequence owns are left as they were; keys outside [0, page_size *
 * max_pages_per_seq) or on a page outside the pool read as zeros.  code * 2^(s - 127) is
 * rounded once, to nearest even: bf16 holds every normal such value exactly; a value past
 * the type's range becomes an infinity.  total == 0 reads nothing.
 */
FA_API fa_status fa_kv_read_paged_fp8(const void *k_pages, const void *v_pages,
                                      const uint8_t *k_scales, const uint8_t *v_scales,
                                      const int32_t *block_table, const int32_t *kv_starts,
                                      const int32_t *cu_seqlens, void *k, void *v, int B, int total,
                                      int Hkv, int D, int num_pages, int page_size,
                                      int max_pages_per_seq, fa_dtype dtype, fa_stream_t stream);

/*
 * Split-KV decode over the 8-bit paged cache, Sq >= 1 query tokens per sequence.
 *   q, o      [B, Sq, Hq, D] (dtype)     lse [B, Hq, Sq] fp32 (may be NULL)
 *   kv_lens   device int32 [B], 0 <= kv_lens[b] <= page_size * max_pages_per_seq; other
 *             values are the caller's error and are clamped on the device
 *   causal    as fa_decode_splitkv_multi: token s sees keys j <= kv_lens[b] - Sq + s
 * (Hq / Hkv) * Sq <= 16; B * Hkv * (page_size * max_pages_per_seq / 64 + 8) < 2^31,
 * B * Sq * Hq <= 2^31 - 9 and Sq * Hq * D <= 2^31 - 256.  A token that sees no key gets O = 0
 * and LSE = -inf.  Cached codes enter the products exactly, queries but for values under 2^-27 of
 * their row's largest, which are off by 2^-38 of it at most.  The factor that makes a sum of
 * products a score, scale * 2^(ks - 127) times a power of two of the query row, is a 32-bit float:
 * where a row's largest |q| times a key's scale passes 2^140 or so it overflows, and a score that
 * would be 0 is NaN.  The probabilities, with V's scales in them, are rounded to fp16 for P.V (11
 * bits for weights down to 2^-25 of the row's largest, fewer below; one under 2^-36 of it may
 * vanish); O is rounded once.  What lies in the pool behind a sequence's last key is not used, nor
 * is a key that `causal` hides from a token used for it, NaN codes there included.  Keys on a page
 * outside the pool count as zero rows.
 *   num_splits  sizes the workspace, which holds B * Hkv * num_splits partial results (<= 0:
 *             fa_decode_default_splits(B, Hkv, page_size * max_pages_per_seq, 0) of a pair).  The
 *             keys of all (sequence, kv head) pairs are laid end to end and cut into equal ranges,
 *             one per CTA that can be resident, but no more than the partial results have room
 *             for, of which r ranges leave at most r + min(r, B * Hkv); where this gives fewer
 *             ranges than pairs to spread, pairs are not cut and a CTA takes whole ones.
 *             1 is taken at its word: no pair is cut, however the lengths differ.  So a caller
 *             who sizes the workspace by fa_decode_default_splits, which answers 1 from eight
 *             pairs an SM up, passes 0 and not that answer: 1280 pairs of 1000 keys but for
 *             eight of 32768 have ranges of 4160 keys with 0, and of 33768 with 1.
 *   workspace at least fa_decode_workspace_bytes(B * Sq, Hq, D, num_splits) bytes (after the
 *             default is applied); no initialisation; not used, and may be NULL, where
 *             num_splits is 1.  Calls that may overlap on the GPU need one each.  A num_splits
 *             for which these bytes pass 2^63 is FA_ERR_UNSUPPORTED.
 * The result does not depend on num_splits beyond rounding; the same inputs give the same
 * bits.
 */
FA_API fa_status fa_decode_splitkv_paged_fp8(const void *q, const void *k_pages, const void *v_pages,
                                             const uint8_t *k_scales, const uint8_t *v_scales,
                                             const int32_t *block_table, const int32_t *kv_lens,
                                             void *o, float *lse, int B, int Sq, int Hq, int Hkv,
                                             int D, int num_pages, int page_size,
                                             int max_pages_per_seq, float scale, int causal,
                                             int num_splits, void *workspace,
                                             size_t workspace_bytes, fa_dtype dtype,
                                             fa_stream_t stream);

/*
 * The 16-bit paged cache, written and attended over.  fa_decode_splitkv_paged reads it; these
 * entry points write it and attend over it with several query tokens, under other masks than
 * "all keys".  The pool is the same:
 *   k_pages, v_pages  [num_pages, page_size, Hkv, D] (dtype)
 *   block_table       device int32 [B, max_pages_per_seq]: key r of sequence b is row
 *                     r % page_size of page block_table[b][r / page_size]
 * D in {64, 96, 128, 256}; B <= 1024; Hkv <= 65536; page_size <= 2^28;
 * page_size * max_pages_per_seq <= 2^31 - 4096.  Table entries outside [0, num_pages) that a call
 * meets are the caller's error: nothing is read or written outside the pool.  Outputs and the
 * workspace must not overlap the inputs, but for q_out below.
 *
 * fa_kv_append_paged_rope writes new rows, keys and queries turned by their positions on the way.
 *   q, k_new, v_new  token t, head h at element t * q_stride (k_stride, v_stride) + h * D, so the
 *                    rows may lie inside a fused projection's output; strides in elements,
 *                    multiples of 8, at least Hq * D (Hkv * D); 16-byte aligned
 *   q_out            [total_new, Hq, D]: the turned queries; may be q where q_stride is Hq * D.
 *                    Hq == 0: no queries, and q and q_out are not used
 *   cu_seqlens_new   device int32 [B + 1]: sequence b's new tokens are packed rows
 *                    [cu_seqlens_new[b], cu_seqlens_new[b + 1]), non-decreasing, ending at most at
 *                    total_new; rows of no sequence are neither written to the pool nor to q_out.
 *                    NULL: every sequence has total_new / B new tokens (B must divide total_new)
 *   kv_lens          device int32 [B]: sequence b's keys INCLUDING the new ones, which become its
 *                    last keys, kv_lens[b] - n .. kv_lens[b] - 1
 *   positions        device int32 [total_new]; NULL: a token's position is its key.  (Drafts of a
 *                    tree, several of which have one position, need them.)
 *   cos, sin         device fp32 [max_pos, rot_dim / 2], 16-byte aligned: of the angles of each
 *                    position.  Positions outside [0, max_pos) are the caller's error and clamped
 *   rot_dim          the first dims of a row that turn: a multiple of 16, 0 .. D (0: none; cos and
 *                    sin may then be NULL); dims from there on are copied
 *   interleaved      zero: pairs (d, d + rot_dim / 2); nonzero: pairs (2 d, 2 d + 1).  A pair
 *                    (x, y) becomes (x cos - y sin, y cos + x sin), in fp32, rounded once
 * Any page_size >= 1.  V's rows are copied.  Rows whose key is outside [0, page_size *
 * max_pages_per_seq) or whose page is outside the pool are dropped (their queries are still
 * written).  total_new == 0 writes nothing.  Two tokens that name one row of a page are the
 * caller's error.  total_new * (Hq + 2 Hkv) < 2^31.
 */
FA_API fa_status fa_kv_append_paged_rope(const void *q, const void *k_new, const void *v_new,
                                         int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                         void *q_out, const int32_t *cu_seqlens_new,
                                         const int32_t *block_table, const int32_t *kv_lens,
                                         const int32_t *positions, const float *cos,
                                         const float *sin, void *k_pages, void *v_pages, int B,
                                         int total_new, int Hq, int Hkv, int D, int rot_dim,
                                         int interleaved, int max_pos, int num_pages, int page_size,
                                         int max_pages_per_seq, fa_dtype dtype, fa_stream_t stream);

/*
 * Bytes of workspace of the two decodes below: two partial results for each SM, of at most 256
 * query rows each, whatever the lengths.  num_sms <= 0 queries the current device.  0 for invalid
 * sizes, or when no device can be queried.
 */
FA_API size_t fa_decode_paged_workspace_bytes(int B, int Sq, int Hq, int Hkv, int D, int num_sms);

/*
 * Attention of a tree of drafted tokens: Sq query tokens per sequence, which are the last Sq keys
 * of its cache (appended before).  Draft t of sequence b is key kv_lens[b] - Sq + t; token i sees
 * every key before the drafts, and draft t where bit t % 32 of word t / 32 of its mask is set.
 *   q, o       [B, Sq, Hq, D] (dtype)     lse [B, Hq, Sq] fp32 (may be NULL)
 *   tree_mask  device int32 [B, Sq, ceil(Sq / 32)]; a token sees itself only if its own bit is
 *              set; bits from Sq on are not used.  Trees of fewer than Sq drafts are padded with
 *              drafts that no mask names (their outputs are computed and meaningless)
 *   kv_lens    device int32 [B], 0 <= kv_lens[b] <= page_size * max_pages_per_seq, clamped on the
 *              device.  Where kv_lens[b] < Sq the drafts before the first key do not exist
 *   workspace  at least fa_decode_paged_workspace_bytes(...) bytes; no initialisation.  Calls that
 *              may overlap on the GPU need one each
 * page_size is a multiple of 16; Sq <= 256; Hq / Hkv <= 128; scale > 0, else FA_ERR_INVALID_ARG.
 * Sq * Hq * D and B * Sq * Hq are below 2^31, and so are the tiles that a plan may have to count: at
 * most B * Hkv * ceil(Sq * Hq / Hkv / 64) * (capacity / 64 + 8), by capacities and not by lengths;
 * past them FA_ERR_UNSUPPORTED.
 * A token that sees no key gets O = 0
 * and LSE = -inf.  What lies in the pool behind a sequence's last key, and a key hidden from a
 * token, is not used for it, NaN and infinities included.  Keys on a page outside the pool count
 * as zero rows.  Accumulation is fp32; P is rounded to the input dtype before the P.V product; O is
 * rounded once.  The same inputs give the same bits.
 */
FA_API fa_status fa_decode_splitkv_paged_tree(const void *q, const void *k_pages,
                                              const void *v_pages, const int32_t *block_table,
                                              const int32_t *kv_lens, const int32_t *tree_mask,
                                              void *o, float *lse, int B, int Sq, int Hq, int Hkv,
                                              int D, int num_pages, int page_size,
                                              int max_pages_per_seq, float scale, void *workspace,
                                              size_t workspace_bytes, fa_dtype dtype,
                                              fa_stream_t stream);

/*
 * Decode with a sliding window and sinks: Sq query tokens per sequence, the last ones of its
 * cache.  Token i, at key p = kv_lens[b] - Sq + i, sees the keys j <= p with
 *     j >= p - window_left    or    j < sinks;
 * window_left == -1 leaves the window unbounded: a causal decode, and for one token the same as
 * fa_decode_splitkv_paged, within 2 % of its time for long sequences and faster for short ones, from
 * pages of any multiple of 16.  The table entries of pages that hold no visible key may be anything
 * (of these only pages that share 32 aligned keys with a visible one are read at all).
 * window_left >= -1 and sinks >= 0, else FA_ERR_INVALID_ARG; everything else as
 * fa_decode_splitkv_paged_tree.
 */
FA_API fa_status fa_decode_splitkv_paged_window(const void *q, const void *k_pages,
                                                const void *v_pages, const int32_t *block_table,
                                                const int32_t *kv_lens, void *o, float *lse, int B,
                                                int Sq, int Hq, int Hkv, int D, int num_pages,
                                                int page_size, int max_pages_per_seq, float scale,
                                                int window_left, int sinks, void *workspace,
                                                size_t workspace_bytes, fa_dtype dtype,
                                                fa_stream_t stream);

/* Static, human-readable name of a status code. */
FA_API const char *fa_status_string(fa_status s);

/*
 * Reads and clears the sticky device status word of the current device that kernels
 * write when a bounded wait gives up (FA_ERR_TIMEOUT); FA_OK if none did.  Synchronises
 * the current device.  FA_ERR_CUDA if the device cannot be queried.
 */
FA_API fa_status fa_last_device_status(void);

/*
 * Self-test of the bounded-wait path that every kernel's barrier waits use.  Enqueues one
 * CTA of two warps on `stream`.  Warp 0 waits on an mbarrier phase that no thread
 * completes.  After the wait limit (2 s of GPU time) it gives up, records FA_ERR_TIMEOUT in
 * the device status word and raises the CTA's abort flag.  Warp 1 starts the same kind of
 * wait 0.5 s later and leaves when it sees the flag.  Nothing faults: every wait ends by
 * itself, and the context stays usable.
 *   result  device int32[3], caller-owned, 16-byte aligned.  It receives:
 *           [0] 1 if warp 0's wait gave up;
 *           [1] 1 if warp 1 left on the abort flag before its own limit;
 *           [2] warp 0's wait in milliseconds.
 * Read the status afterwards with fa_last_device_status(), which also clears it.
 * FA_ERR_INVALID_ARG for a null or misaligned result; FA_ERR_CUDA if the launch failed.
 */
FA_API fa_status fa_selftest_bounded_wait(int *result, fa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_H_ */
