/*
 * w4_step.h -- C ABI of the decode step's operators between and behind its
 * 4-bit linears (MI355X, gfx950): a paged cache that holds keys and values in
 * 4 bits, what fills it, the attention that reads it, and the sampler that
 * reads the logits.  Part of the same library as w4.h, with its conventions:
 * the caller owns every buffer, arguments are validated on the host before
 * any HIP call, calls are asynchronous on ``stream``, never allocate, never
 * synchronise and can be captured into a HIP graph; an empty problem is
 * W4_OK with nothing launched, and an array without elements may be NULL; the
 * same call on the same inputs returns the same bits.  Outputs must not overlap any input unless said otherwise.
 *
 * The cache.  Pages of ``block_size`` tokens, each with every key/value head;
 * a slot is page * block_size + offset.  A token's vector of one head is cut
 * into groups of G = min(head_dim, 128) values; each group has an FP16 scale
 * s and an FP16 minimum m, and its codes are the library's INT4 nibbles
 * (bits 4j..4j+3 of word p hold d = 8p + j):
 *   x[d] = q[d] * s + m
 *   k_codes int32 [num_blocks][kv_heads][block_size][head_dim/8]
 *   v_codes int32 [num_blocks][kv_heads][block_size/4][head_dim/8][4]
 *           (last axis: token % 4; four tokens' words of one place are one
 *           16-byte load, the shape in which the product with the weights of
 *           the softmax wants them)
 *   k_meta, v_meta fp16 [num_blocks][kv_heads][head_dim/G][block_size][2]   (s, m)
 * What a quantised group stores, from its BF16 values x (magnitudes above
 * 65504 count as 65504):
 *   s = fp16((max - min) * fp32(1/15)), m = fp16(min),
 *   q = clamp(rint((x - m) * fp32(1/s)), 0, 15), all 0 where s = 0
 * in FP32; a group that holds an infinity or a NaN stores s = NaN, so that
 * whatever reads it is NaN.
 * Slots may pass any 32-bit byte offset: addresses are formed in 64 bits.
 */
#ifndef W4_STEP_H
#define W4_STEP_H

#include "w4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Pages hold 16, 32, 64, 128 or 256 tokens; heads 64, 128 or 256 values. */
#define W4_KV4_GROUP 128
#define W4_KV4_MIN_BLOCK 16
#define W4_KV4_MAX_BLOCK 256

typedef struct w4_kv4_cache {
    void* k_codes; /* device int32, 16-byte aligned (all four) */
    void* k_meta;  /* device fp16 */
    void* v_codes; /* device int32 */
    void* v_meta;  /* device fp16 */
    int num_blocks;
    int block_size;
    int kv_heads;
    int head_dim;
} w4_kv4_cache;

/*
 * w4_kv4_plan -- block tables, slot map, positions and row ranges of a step,
 * from the requests' lengths.
 *   cached, new_tokens  device int32 [B]: tokens a request holds in the cache
 *                       already, and those this step adds (0: it rests;
 *                       negative counts as 0)
 *   block_table  device int32 [B][max_blocks], in and out: entries of the
 *                ceil(cached / block_size) pages a request holds are read,
 *                entries of the pages it needs besides are written, nothing
 *                else is touched
 *   free_blocks  device int32 [free_capacity]: a stack of free pages, of
 *                which free_count (device int32 [1], clamped into
 *                [0, free_capacity]) are left.  The r-th page that the step
 *                needs (requests in order, each one's pages in order) gets
 *                free_blocks[free_count - 1 - r], or -1 where none is left
 *   q_start      device int32 [B+1], out: first row of each request, the sum last
 *   kv_lens      device int32 [B], out: cached + new_tokens
 *   positions, slots  device int32 [rows], out: for each row its token's
 *                position in its request and its slot.  A token without a
 *                page (none left, past max_blocks, or a negative entry) has
 *                slot -1; rows behind the last request have -1 in both
 *   counts       device int32 [2], out: pages left on the stack, pages that
 *                were short.  The caller moves on by passing counts[0] as the
 *                next free_count.
 *   0 <= B <= W4_KV4_PLAN_MAX_BATCH; block_size a power of two in
 *   [1, 4096]; sums of lengths stay below 2^31 (larger ones saturate).
 * B = 0 writes q_start, the padding and counts.
 * Outputs must not overlap each other or an input.
 * Errors: W4_ERR_NULL, W4_ERR_SHAPE, W4_ERR_ALIGN, W4_ERR_ALIAS, W4_ERR_ARG, W4_ERR_HIP.
 */
#define W4_KV4_PLAN_MAX_BATCH 4096
W4_API w4_status w4_kv4_plan(const int32_t* cached, const int32_t* new_tokens, int32_t* block_table,
                             const int32_t* free_blocks, const int32_t* free_count, int B, int max_blocks,
                             int free_capacity, int block_size, int rows, int32_t* q_start, int32_t* kv_lens,
                             int32_t* positions, int32_t* slots, int32_t* counts, void* stream);

/*
 * w4_qk_norm_rope -- RMS norm of each query and key head, rotation by
 * position, and (with a cache) keys and values quantised into it, in one pass.
 *   y = x / sqrt(mean(x^2) + eps) * (weight + weight_add)     (no weight: y = x)
 *   (y_i, y_j) -> (y_i cos - y_j sin, y_j cos + y_i sin) for the pairs
 *   (i, j) = (i, i + rot_dim / 2), or (2i, 2i + 1) if interleaved,
 *   i < rot_dim / 2; values from rot_dim on are not rotated
 * Norm and rotation are in FP32 for queries (in FP64 for a head whose mean
 * square lies outside 2^-40 .. 2^40, and for weights from 2^60 on) and FP64 for
 * keys (whose result decides a code); each result is rounded to BF16, one from
 * FP64 to FP32 before that.  The cache takes the rounded key and the value as given.
 *   q, k, v      device bf16 [T][heads][head_dim], 16-byte aligned; rows
 *                *_stride elements apart (a multiple of 8, at least
 *                heads * head_dim), so the three may lie side by side.
 *                q may be NULL if q_heads = 0; v only with a cache
 *   q_weight, k_weight  device bf16 [head_dim], 16-byte aligned, or NULL
 *   cos_sin      device float [max_pos][rot_dim], 16-byte aligned: a row's
 *                rot_dim / 2 cosines, then its sines; NULL if rot_dim = 0
 *   positions    device int32 [T]; NULL if rot_dim = 0.  A row with a
 *                negative position is padding: nothing is written for it.  A
 *                position of max_pos or more makes its q and k NaN
 *   slots        device int32 [T], with a cache: where each row's key and
 *                value go; nothing is stored for one outside the cache.  The
 *                slots of one call that lie in the cache must differ
 *   q_out, k_out device bf16, layouts as q and k with their own strides.
 *                Each may be exactly its input (same pointer and stride).
 *                k_out may be NULL with a cache
 *   rot_dim      a multiple of 16 in [0, head_dim]
 *   T            at most 2^26 - 4
 *   cache        NULL, or the cache (its kv_heads and head_dim are used)
 * Errors: W4_ERR_NULL, W4_ERR_SHAPE, W4_ERR_UNSUPPORTED (head_dim, block
 * size), W4_ERR_ALIGN, W4_ERR_ALIAS, W4_ERR_ARG (strides, rot_dim, eps), W4_ERR_HIP.
 */
typedef struct w4_qk_args {
    const void* q;
    const void* k;
    const void* v;
    int64_t q_stride, k_stride, v_stride; /* elements */
    const void* q_weight;
    const void* k_weight;
    const float* cos_sin;
    const int32_t* positions;
    const int32_t* slots;
    void* q_out;
    void* k_out;
    int64_t q_out_stride, k_out_stride;
    int T, q_heads, kv_heads, head_dim;
    int rot_dim, max_pos, interleaved;
    float eps, weight_add;
} w4_qk_args;
W4_API w4_status w4_qk_norm_rope(const w4_qk_args* args, const w4_kv4_cache* cache, void* stream);

/*
 * w4_kv4_read -- the keys and values that the cache stands for.
 *   slots         device int32 [n]; a row whose slot lies outside the cache is
 *                 not written
 *   k_out, v_out  device bf16 [n][kv_heads][head_dim], 16-byte aligned:
 *                 bf16(q * s + m); either may be NULL, not both; at most 2^35 - 2^11
 *                 values in each
 * Errors: W4_ERR_NULL, W4_ERR_SHAPE, W4_ERR_UNSUPPORTED, W4_ERR_ALIGN, W4_ERR_ALIAS, W4_ERR_HIP.
 */
W4_API w4_status w4_kv4_read(const w4_kv4_cache* cache, const int32_t* slots, int n, void* k_out, void* v_out,
                             void* stream);

/*
 * w4_kv4_attn -- attention of each request's new rows over its cached tokens.
 *   out[t][h] = sum_j p_j v_j,  p = softmax over the visible j of scale * q[t][h] . k_j
 * Request b owns rows q_start[b] .. q_start[b+1] - 1 (or row b alone if
 * q_start is NULL; then T = B); its row i stands at position
 * pos = kv_lens[b] - rows(b) + i and sees the tokens
 *   j <= pos  and  (window = 0, or j > pos - window, or j < sinks).
 * The tokens are already in the cache (their own included).  Query head h
 * reads key/value head h / (q_heads / kv_heads).  A row that sees nothing is 0.
 * Scores, softmax statistics and sums are FP32; a weight times a value's
 * scale is rounded to two BF16 parts (2^-16 of it), the result once to BF16.
 * How the work is cut goes by max_q, B and max_kv alone: requests of one new
 * token beside long prompts are faster in a call of their own.
 *   q            device bf16 [T][q_heads][head_dim], 16-byte aligned, rows
 *                q_stride elements apart (a multiple of 8)
 *   block_table  device int32 [B][max_blocks]: a row that sees a token whose
 *                entry lies outside [0, num_blocks) or past max_blocks is NaN
 *                (nothing is read for it); other entries are not used
 *   kv_lens      device int32 [B] (negative counts as 0)
 *   q_start      device int32 [B+1], clamped into [0, T]; a request's end below
 *                its start counts as empty.  Rows in no request are not written
 *   max_q        the most rows of any request: its rows past max_q are not
 *                written (precondition, not checked)
 *   max_kv       about the most cached tokens of any request: only the work's
 *                split goes by it, any value is correct
 *   out          device bf16 [T][q_heads][head_dim], 16-byte aligned, rows
 *                out_stride elements apart
 *   workspace    at least w4_kv4_attn_workspace_bytes() bytes for the same
 *                arguments (NULL when that is 0), 16-byte aligned: partial
 *                sums of a split work.  Its contents on entry are ignored.
 *                Calls that share one workspace must be ordered
 *   q_heads a multiple of the cache's kv_heads; scale > 0 and finite;
 *   window, sinks >= 0.
 * Errors: W4_ERR_NULL, W4_ERR_SHAPE, W4_ERR_UNSUPPORTED (head_dim, block
 * size), W4_ERR_ALIGN, W4_ERR_WORKSPACE, W4_ERR_ALIAS, W4_ERR_ARG, W4_ERR_HIP.
 */
typedef struct w4_attn_args {
    const void* q;
    void* out;
    int64_t q_stride, out_stride; /* elements */
    const int32_t* block_table;
    const int32_t* kv_lens;
    const int32_t* q_start;
    int T, B, q_heads, max_blocks;
    int max_q, max_kv;
    int window, sinks;
    float scale;
} w4_attn_args;
/* Only T, B, q_heads, max_q, max_kv, window and sinks, and the cache's kv_heads and head_dim are read. */
W4_API size_t w4_kv4_attn_workspace_bytes(const w4_attn_args* args, const w4_kv4_cache* cache);
W4_API w4_status w4_kv4_attn(const w4_attn_args* args, const w4_kv4_cache* cache, void* workspace,
                             size_t workspace_bytes, void* stream);

/*
 * w4_sample -- one token from each row of logits, from a given uniform number.
 * Over a row's tokens in the order (logit falling, index rising):
 *   weight w = exp((logit - largest) / temperature)
 *   kept: the first top_k, of these the shortest beginning whose weight
 *   reaches top_p of theirs, of these the ones with w >= min_p; the first
 *   token always.  The result is the first kept token at which the running
 *   weight exceeds uniform * (the kept weight).
 * Weights and sums are FP64.  -0 and +0 are equal; NaN counts as -infinity; a
 * row of nothing but these gives -1; beside a +infinity everything less has
 * weight 0.
 *   logits       device bf16 [rows][vocab], rows row_stride elements apart, 2-byte aligned
 *   uniform      device double [rows] in [0, 1); less counts as 0, above 1 - 2^-40 as
 *                that, so that no rounding of the sums draws a token without weight
 *   temperature  device float [rows] (not above 0: the largest logit), or NULL for 1
 *   top_k        device int32 [rows] (0 or less: all), or NULL
 *   top_p        device float [rows] (1 or more: all), or NULL
 *   min_p        device float [rows] (0 or less: all), or NULL
 *   tokens       device int32 [rows], out
 *   workspace    at least w4_sample_workspace_bytes(rows, vocab) bytes, 16-byte
 *                aligned (NULL when that is 0); contents ignored on entry;
 *                calls that share one must be ordered
 *   1 <= vocab <= W4_SAMPLE_MAX_VOCAB, rows >= 0
 * Errors: W4_ERR_NULL, W4_ERR_SHAPE, W4_ERR_ALIGN, W4_ERR_WORKSPACE, W4_ERR_ALIAS, W4_ERR_ARG, W4_ERR_HIP.
 */
#define W4_SAMPLE_MAX_VOCAB 1048576
W4_API size_t w4_sample_workspace_bytes(int rows, int vocab);
W4_API w4_status w4_sample(const void* logits, int64_t row_stride, const double* uniform, const float* temperature,
                           const int32_t* top_k, const float* top_p, const float* min_p, int32_t* tokens, int rows,
                           int vocab, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W4_STEP_H */
