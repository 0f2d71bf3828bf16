/*
 * kv8.h -- C ABI of a paged key/value cache held in 8 bits with one float32
 * scale for each page and head, and of the attention that reads it.
 *
 * Cache. A page holds P tokens of every key/value head (P = 16, 32, 64, 128
 * or 256), D = 64, 128 or 256 values a token and head:
 *   k_codes  [pages][Hkv][P][D]   one byte each: int8 (KV8_INT8) or e4m3 (KV8_E4M3)
 *   v_codes  [pages][Hkv][D][P]   a head's page is stored transposed: the product with the
 *                                 probabilities runs along the tokens, which are then contiguous
 *   k_scale, v_scale [pages][Hkv] float32, finite, not negative; a value is code * scale (codes under scale 0 are 0)
 *   page_table [B][max_pages] int32: token t of sequence b lies in page page_table[b][t / P], slot t % P
 * Sequences may share pages that none of them appends to. Entries outside
 * 0 .. pages - 1 hold no tokens: appending there stores nothing, reading gives
 * zeros, attention leaves the tokens out.
 *
 * Packed tokens. The tokens of a call (queries, or new keys and values) lie
 * packed, those of sequence b at rows cu[b] .. cu[b+1] - 1 (cu [B + 1] int32,
 * cu[0] = 0, not decreasing, cu[B] = total); they are the LAST tokens of the
 * sequence, whose length kv_len[b] (int32) counts them in: with n of them, the
 * i-th stands at position kv_len[b] - n + i. max_new bounds n; a sequence with
 * more is refused nothing, but only its first max_new tokens are handled.
 * Lengths above max_pages * P count as max_pages * P. Row r of a packed tensor
 * starts at r * stride elements (stride >= heads * D), its heads are contiguous.
 *
 * Conventions (pointers, streams, workspaces, statuses) are those of q4.h.
 */
#ifndef KV8_H
#define KV8_H

#include <stddef.h>
#include <stdint.h>

#include "q4.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { KV8_INT8 = 0, KV8_E4M3 = 1 };

/* The cache and the sequences of a call. */
typedef struct {
    int format;        /* KV8_INT8 or KV8_E4M3 */
    int pages;         /* pages in the cache */
    int kv_heads;      /* Hkv */
    int page_size;     /* P */
    int head_dim;      /* D */
    int batch;         /* B */
    int max_pages;     /* entries in a row of page_table */
    void* k_codes;     /* 16-byte aligned */
    void* v_codes;     /* 16-byte aligned */
    float* k_scale;
    float* v_scale;
    const int32_t* page_table;
    const int32_t* kv_len;   /* [B] */
    const int32_t* cu;       /* [B + 1] */
} kv8_cache;

/*
 * Stores the packed new keys and values (dtype Q4_DT_F32 or Q4_DT_BF16). For every page and head that gets tokens:
 *   s_new = max|x| of its new tokens / L   (L = 127 for int8, 448 for e4m3; float32, correctly rounded)
 *   s     = s_new if the page's first new token is in slot 0, else max(the page's scale, s_new)
 *   codes of tokens that the page held before: round(c * (s_old / s)) where s grew (s_old / s and the product in
 *   float32), unchanged otherwise; new codes: round(x / s) with the float32 quotient, cut at +-L; 0 where s is 0
 * (round: half to even, to an integer or to an e4m3 value). A NaN is stored as 0, an infinity as the largest finite
 * float32: codes and scales stay finite. (The page's scale is then 2^120 or so, under which ordinary values are 0.)
 */
int kv8_append(const kv8_cache* cache, int total, int max_new, int dtype, const void* k_new, long long k_stride,
               const void* v_new, long long v_stride, void* stream);

/* Writes the values (code * scale, in dtype) of the last n tokens of each sequence, packed as above:
 * k_out, v_out [total][Hkv][D], contiguous, 16-byte aligned. Rows of positions below 0 are zero. */
int kv8_read(const kv8_cache* cache, int total, int max_new, int dtype, void* k_out, void* v_out, void* stream);

/* Bytes of the workspace of kv8_attention (0 for sizes that it refuses). max_kv bounds the lengths. */
size_t kv8_attention_work_bytes(const kv8_cache* cache, int total, int max_new, int max_kv, int heads);

/*
 * Attention of the packed queries q [total][heads][D] (dtype Q4_DT_F32 or Q4_DT_BF16) over the cache, heads a
 * multiple of Hkv (query head h reads key/value head h / (heads / Hkv)):
 *   out[r][h] = sum_t p_t v_t,  p = softmax_t(scale * q . k_t)
 * over the positions t <= that of the query, with window > 0 only the last `window` of them, and t < max_kv. A query
 * that sees no key gives zeros. out [total][heads][D] in q's dtype, contiguous. lse [total][heads] float32 may be
 * NULL: log(sum_t exp(scale * q . k_t)), -infinity for a query that sees no key. A query with a NaN gives NaN in both.
 * Softmax statistics and sums are float32, and codes enter the products exactly. A token's weight is p_t times its
 * page's value scale. For float32 results queries enter as two f16 halves (22 bits of the row's largest value) and
 * weights in full. For bfloat16 results queries are exact (22 bits of the row's largest value) and a weight is rounded
 * to f16's eleven bits, or to 2^-36 of the row's largest weight (to 2^(k - 36) of it where no value scale is above
 * 2^(-80 - k)): a page whose value scale is 2^36 times another's hides that one's values.
 */
int kv8_attention(const kv8_cache* cache, int total, int max_new, int max_kv, int heads, int dtype, const void* q,
                  long long q_stride, float scale, int window, void* out, float* lse, void* work, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KV8_H */
