/*
 * latent_attn.h -- C ABI of the paged latent cache and of the attention that
 * reads it on GB300 (sm_103a).
 *
 * The output of this attention is what invrope_postmix_fwd (invrope.h) takes:
 * one latent vector c_t of d = nope + pe channels a token serves as key AND
 * value of every head, so the output's trailing pe channels still carry the
 * keys' rotation, which the postmix undoes. The index tables of the sparse
 * form are those kv_idx_local_to_global (invrope.h) makes.
 *
 * Cache: `num_slots` rows of kv_latent_row_bytes() bytes, back to back, at a
 * 16-byte aligned address; slot s is row s. A page is `page_size` consecutive
 * slots (any size >= 1), page g being slots g*page_size .. +page_size-1.
 *
 *   KV_LATENT_BF16 : d bf16 values.
 *   KV_LATENT_E4M3 : nope e4m3 codes, pe bf16 values, ceil(nope/64) scale
 *       bytes, padding to a multiple of 16 bytes (left as it was). A scale byte
 *       b stands for 2^(b-127) and belongs to 64 consecutive channels (fewer
 *       in the last group); a channel's value is code * 2^(b-127), rounded
 *       once to bf16. b = 255 makes its whole group read as NaN.
 *       kv_latent_write stores scale bytes 7 to 246 and 255, with which values
 *       are exact in bf16. Rows that another program wrote may hold any byte:
 *       below 7 a value may round in bf16's subnormals, above 246 it may be an
 *       infinity, in kv_latent_read and in the attention alike. The codes 0x7F
 *       and 0xFF, NaN in other uses of e4m3, are no NaN in a row: both calls
 *       take them as 480 and -480, which follow 448. kv_latent_write stores
 *       neither; a program that writes rows itself and has a NaN to store has
 *       the scale byte 255 for it.
 *
 * Common contract, beside that of invrope.h (device pointers of the current
 * device, work enqueued on `stream` only, arguments checked on the host before
 * anything is enqueued, the same status codes, no allocation, bounded waits
 * that report through invrope_take_device_fault):
 *   - pe >= 0 and nope >= 0, d = nope + pe >= 8 a multiple of 8; for
 *     KV_LATENT_E4M3 nope >= 16 a multiple of 16 and pe a multiple of 8
 *     (else INVROPE_ERR_INVALID_ARG). d <= 512 (else INVROPE_ERR_UNSUPPORTED).
 *   - 1 <= num_slots < 2^31 (else INVROPE_ERR_INVALID_ARG / _UNSUPPORTED). Row addresses are
 *     computed in 64 bits.
 *   - Slots, pages, indices and lengths lie in device memory, so they are
 *     checked by the kernels: what is out of range is never followed. Each
 *     call says what it does instead.
 */
#ifndef LATENT_ATTN_H_
#define LATENT_ATTN_H_

#include <stddef.h>
#include <stdint.h>

#include "invrope.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KV_LATENT_BF16 0
#define KV_LATENT_E4M3 1

/* Bytes of one cache row; 0 when nope, pe or fmt is invalid. */
size_t kv_latent_row_bytes(int nope, int pe, int fmt);

/*
 * Store n tokens' latent vectors, quantising them where the cache is 8-bit:
 *
 *   cache[slots[i]] = x[i]                                    (KV_LATENT_BF16)
 *   for each group of 64 channels: e the least whole number with
 *   amax <= 448 * 2^e, kept to [-120, 119];
 *   code = e4m3(x * 2^-e), to nearest even, magnitudes over 448 to 448;
 *   scale byte e + 127                                        (KV_LATENT_E4M3)
 *
 * A group that holds an infinity or a NaN gets the scale byte 255. The pe
 * channels keep their bf16 bits.
 * x     : bf16 [n, d], 16-byte aligned. slots : int32 [n], 4-byte aligned.
 * cache : must overlap neither. n >= 0 (0 enqueues nothing), below 2^31 (else
 * INVROPE_ERR_UNSUPPORTED; kv_latent_read too).
 * A slot outside [0, num_slots) stores nothing. Two equal slots in one call
 * leave that row undefined.
 */
int kv_latent_write(const void* x, const int32_t* slots, void* cache,
                    int64_t n, int64_t num_slots, int nope, int pe, int fmt,
                    struct CUstream_st* stream);

/*
 * Read rows back: out[i] = value of cache[slots[i]] (bf16 [n, d], exact); a
 * slot outside [0, num_slots) gives zeros. out : 16-byte aligned, overlaps
 * neither input.
 */
int kv_latent_read(const void* cache, const int32_t* slots, void* out,
                   int64_t n, int64_t num_slots, int nope, int pe, int fmt,
                   struct CUstream_st* stream);

/*
 * Workspace bytes of the two attention calls on the CURRENT device for rows
 * query rows of nh heads, where a row attends to at most max_tokens tokens
 * (max_pages * page_size, or topk). 0 when no row can be split (then the
 * workspace may be NULL) or when an argument is invalid.
 */
size_t latent_attn_workspace_bytes(int64_t rows, int nh, int64_t max_tokens,
                                   int nope, int pe);

/*
 * Attention of one new token a row over its pages:
 *
 *   s[r,h,t]  = scale * q[r,h,:] . c(r,t)     t < lens[r]
 *   O[r,h,:]  = sum_t softmax_t(s[r,h,:]) c(r,t)
 *   lse[r,h]  = log sum_t exp s[r,h,t]
 *   c(r,t)    = value of cache slot page_table[r, t / page_size] * page_size
 *               + t % page_size
 *
 * q    : bf16 [rows, nh, d], O : bf16 [rows, nh, d], 16-byte aligned.
 * lse  : fp32 [rows, nh] or NULL.
 * page_table : int32 [rows, max_pages]; lens : int32 [rows].
 * cache: num_pages pages of page_size slots; num_pages * page_size < 2^31 and
 *      max_pages * page_size < 2^31 (else INVROPE_ERR_UNSUPPORTED).
 * workspace : 16-byte aligned scratch of at least
 *      latent_attn_workspace_bytes(rows, nh, max_pages * page_size, nope, pe)
 *      bytes; its contents on entry do not matter. Calls that overlap on the
 *      GPU need one each.
 * O, lse and the workspace's bytes that the call needs overlap neither each other
 * nor an input (else INVROPE_ERR_INVALID_ARG).
 * rows >= 0, 1 <= nh <= 128 (above: INVROPE_ERR_UNSUPPORTED), rows * nh < 2^31,
 * scale * log2(e) within fp32's range (else INVROPE_ERR_INVALID_ARG).
 * Several new tokens of one sequence are several rows: repeat its page list
 * and give each its own length.
 * lens[r] is taken as 0 where negative and as max_pages * page_size where
 * larger. Tokens of a page outside [0, num_pages) are left out. A row that
 * attends to nothing gets O = 0 and lse = -inf. Cache rows that are not
 * attended to are not read, so their contents (NaN too) do not matter; an
 * infinity or a NaN in an attended row or in q shows in the heads it reaches;
 * a head whose scores are all -inf gets O = NaN and lse = -inf.
 * Scores, sums and accumulators are fp32; the weights are rounded once to
 * bf16 for the second product and O once to bf16. For given arguments and
 * device memory contents the results have the same bits on every call.
 */
int latent_attn_decode(const void* q, const void* cache, const int32_t* page_table,
                       const int32_t* lens, void* O, float* lse,
                       void* workspace, size_t workspace_bytes,
                       int64_t rows, int nh, int nope, int pe, int fmt,
                       int64_t num_pages, int page_size, int64_t max_pages,
                       double scale, struct CUstream_st* stream);

/*
 * The same attention over the cache rows that an index table selects: row r
 * attends to slots idx[r, 0..topk-1]. An index outside [0, num_slots) is left
 * out (kv_idx_local_to_global keeps padding negative); one that appears twice
 * counts twice. idx : int32 [rows, topk], 4-byte aligned, 0 <= topk < 2^31 (above:
 * INVROPE_ERR_UNSUPPORTED).
 * workspace : latent_attn_workspace_bytes(rows, nh, topk, nope, pe) bytes.
 * Everything else as in latent_attn_decode.
 */
int latent_attn_sparse(const void* q, const void* cache, const int32_t* idx,
                       void* O, float* lse,
                       void* workspace, size_t workspace_bytes,
                       int64_t rows, int nh, int nope, int pe, int fmt,
                       int64_t num_slots, int64_t topk,
                       double scale, struct CUstream_st* stream);

#ifdef __cplusplus
} /* extern "C" */
#endif

#endif /* LATENT_ATTN_H_ */
