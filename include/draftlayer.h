/*
 * draftlayer.h -- C ABI of the draft layer's attention for MI355X (gfx950),
 * in the same library as the draft head (drafthead.h).
 *
 * Before a draft slot's hidden row reaches the head it passes the draft
 * layer's attention: queries and keys are rotated by their positions, keys
 * and values are put into a paged cache held in 8 bits, and the queries attend
 * over that cache.  The projections around it are plain library products and
 * stay with the caller.
 *
 * Call sequence:
 *   load time (host):  draft_layer_rope_table -> copy to device
 *   per step (device): draft_layer_append -> draft_layer_attend
 *   for a caller that wants the cached values in bf16: draft_layer_read
 *
 * The conventions are drafthead.h's: DH_OK or a negative DH_E* code, nothing
 * thrown, every argument checked before any HIP call, the caller owns every
 * buffer, device functions enqueue on `stream` and return,
 * draft_head_last_error() describes the last error of the calling thread.
 *
 * A batch (all device functions): n_seq sequences with T rows of new tokens.
 *   q_start  device, int32 [n_seq + 1], not decreasing, 0 first, at most T:
 *            rows q_start[s] .. q_start[s+1] - 1 are sequence s's new tokens
 *            (n_s of them, 0 allowed)
 *   kv_len   device, int32 [n_seq]: tokens of sequence s in the cache, its new
 *            ones included; row i of s is the token at position
 *            kv_len[s] - n_s + i.  Rows of negative positions have no token.
 *            Rows from q_start[n_seq] on belong to no sequence: draft_layer_read
 *            and draft_layer_attend leave their outputs as they are, and what
 *            draft_layer_append puts into their q_out is of no use.
 *   table    device, int32 [n_seq][max_pages]: page ids, page j of a sequence
 *            holding positions j*page .. j*page + page - 1.  Entries beyond a
 *            sequence's length are not used.  Positions from max_pages*page
 *            on do not exist: nothing is written there and nothing seen.
 *            An id outside 0 .. n_pages - 1 is treated the same way.
 *
 * The cache: per page and key/value head, page*D codes for keys and for values
 * and one fp32 scale each; a code byte u stands for (u - 128) * scale.
 *   k_codes, v_codes  device, uint8 [n_pages][hkv][page*D], 16-byte aligned
 *   k_scale, v_scale  device, fp32 [n_pages][hkv]
 * Inside a (page, head) the bytes stand in the order in which the matrix
 * instruction's lanes take them (16 bytes a lane, 1 KiB an instruction): with
 * u = t % 32 for token t of the page and element e of the head,
 *   key    (t/32)*32*D + (((u/16)*(D/64) + e/64)*64 + ((e%64)/16)*16 + u%16)*16 + e%16
 *   value  (t/32)*32*D + (((e/32)*4 + (u%16)/4)*16 + e%16)*16 + ((e%32)/16)*8 + (u/16)*4 + u%4
 * A fresh cache needs no initial contents.
 *
 * Limits (all): D 64, 128 or 256; page 32, 64, 128 or 256; 1 <= hkv <= hq <=
 * DL_MAX_HEADS, hq a multiple of hkv; 0 <= T <= DL_MAX_ROWS; 1 <= n_seq <=
 * DL_MAX_SEQS; max_pages*page < 2^30.  T = 0 does nothing.
 */
#ifndef DRAFTLAYER_H
#define DRAFTLAYER_H

#include "drafthead.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DL_MAX_HEADS 256
#define DL_MAX_ROWS (1 << 22)
#define DL_MAX_SEQS 4096
#define DL_MAX_POSITIONS (1 << 30)
#define DL_WORKSPACE_ZERO_BYTES 6144   /* the start of a workspace that has to be zero before its first use */

/*
 * HOST.  cos and sin of the rotary angles: out[p][i] = (m cos(p f_i),
 * m sin(p f_i)), computed in double and rounded once, for p < positions and
 * i < rot/2, with f_i = base^(-2i/rot) stretched for contexts longer than the
 * trained one:
 *   factor = 1                 f_i as it is
 *   factor > 1, original = 0   f_i / factor (positions interpolated)
 *   factor > 1, original > 0   YaRN's ramp (Peng et al. 2023, "NTK by parts"):
 *     f_i (1 - r_i) + f_i / factor r_i with r_i = clamp((i - lo)/(hi - lo), 0, 1),
 *     lo = max(floor(c(beta_fast)), 0), hi = min(ceil(c(beta_slow)), rot - 1)
 *     (hi - lo at least 0.001), c(n) = rot ln(original / (2 pi n)) / (2 ln base)
 *   out      fp32 [positions][rot/2][2]
 *   mscale   m, the factor on both (1; YaRN recommends 0.1 ln(factor) + 1)
 * Errors: DH_EINVAL (null out; base <= 1, factor < 1, mscale <= 0, original <
 * 0 or beta_fast, beta_slow <= 0, or not finite), DH_ESHAPE (positions < 1 or
 * > DL_MAX_POSITIONS, rot not a positive even number or > 256).
 */
int draft_layer_rope_table(int positions, int rot, double base, double factor, int original, double beta_fast,
                           double beta_slow, double mscale, float* out);

/*
 * DEVICE.  Rotate the new queries and keys, and write the new keys and values
 * to the cache in 8 bits.
 * A rotary pair (a, b) of a head's first rot elements is (x[i], x[i + rot/2]),
 * or (x[2i], x[2i+1]) with interleaved != 0, and becomes (a cos - b sin,
 * b cos + a sin) with rope's entry i of the token's position; the elements
 * from rot on stay.  Every step below is one fp32 operation rounded on its
 * own.  q_out is the rotated query in bf16; the rotated key goes to the cache
 * without another rounding.  For each page that holds a new token, each head,
 * and keys and values on their own:
 *   step = max(amax / 127, 2^-40) over the page's new values, and at least
 *          the present scale if the page holds older tokens of the sequence;
 *   where that raises the scale, an older code c becomes rne(c * (old / step));
 *   a new code is rne(x * (1 / step)) clamped to -127..127; scale = step.
 * A new value that is infinite or NaN (in a key: after the rotation) makes its
 * page's and head's scale NaN, whatever the codes: all tokens of that page read
 * back as NaN, and so is every row that sees one, until the page starts afresh.
 * A page whose first new token is its token 0 starts afresh, whatever its
 * scale and codes held.  Rejected tokens are dropped by writing over them; what
 * one has done to a page that also holds accepted tokens stays: where it raised
 * the scale, the accepted codes are re-rounded to the larger step, and the scale
 * keeps it until the page starts afresh.
 *   q        device, bf16, row r head h at q + r*ldq + h*D; may be NULL with
 *            q_out (keys and values only)
 *   k, v     device, bf16, row strides ldk, ldv
 *   rope     device, fp32 [positions][rot/2][2], positions >= max_pages*page
 *   q_out    out, bf16 [T][hq][D] without gaps; may be q itself if ldq = hq*D
 * Row strides are in elements, multiples of 8 and at least the heads' D each;
 * q, k, v, q_out and rope are 16-byte aligned.  Two sequences of one call
 * must not write the same page.  Values (of q, k and v) below 2^60 in magnitude
 * and rope entries below 4 leave rotated elements below 2^63 and scales below
 * 2^57, which is what draft_layer_attend takes.
 * Limits: rot a multiple of 16 in 0..D (0: nothing is rotated, rope unused).
 * Errors: DH_EINVAL, DH_ESHAPE, DH_EUNSUP, DH_EHIP.
 */
int draft_layer_append(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                       const float* rope, int positions, int rot, int interleaved, uint8_t* k_codes,
                       uint8_t* v_codes, float* k_scale, float* v_scale, int n_pages, int page,
                       const int32_t* q_start, const int32_t* kv_len, const int32_t* table, int n_seq,
                       int max_pages, int T, int hq, int hkv, int D, void* q_out, void* stream);

/*
 * DEVICE.  Read the cache back: row r of sequence s (the batch's rows, at
 * position kv_len[s] - n_s + i) is bf16(code * scale) of its token, rounded to
 * nearest even; zero where there is no token.
 *   k_out, v_out  out, bf16 [T][hkv][D], 16-byte aligned
 * Errors: DH_EINVAL, DH_ESHAPE, DH_EUNSUP, DH_EHIP.
 */
int draft_layer_read(const uint8_t* k_codes, const uint8_t* v_codes, const float* k_scale, const float* v_scale,
                     int n_pages, int page, const int32_t* q_start, const int32_t* kv_len, const int32_t* table,
                     int n_seq, int max_pages, int T, int hkv, int D, void* k_out, void* v_out, void* stream);

/*
 * Bytes of device workspace that draft_layer_attend needs at most for calls of
 * up to T rows of up to n_seq sequences with these heads: one size, asked for
 * the largest batch, serves them all.  Its first DL_WORKSPACE_ZERO_BYTES must
 * be zero before its first use, the rest may hold anything; the calls leave those
 * bytes at zero, so one workspace serves any number of calls in order (one
 * stream), with other heads too where it is large enough for them.
 * Errors: DH_EINVAL (null pointer), DH_ESHAPE, DH_EUNSUP.
 */
int draft_layer_workspace_bytes(int T, int n_seq, int hq, int hkv, int D, size_t* bytes);

/*
 * DEVICE.  Attention of the rows over the cache.  Query head h reads key/value
 * head h / (hq/hkv).  The row at position p sees the cached tokens j <= p
 * and, with window > 0, of these only j > p - window and j < sinks (the first
 * tokens that stay visible).  With z_j = scale q.k_j over the tokens that a
 * row sees:
 *   out  = sum_j exp(z_j - lse) v_j   bf16 [T][hq][D], 16-byte aligned
 *   lse  = ln sum_j exp(z_j)          fp32 [T][hq]; may be NULL
 * A row that sees nothing gets out = 0 and lse = -inf.  Products run on the
 * matrix cores in fp16 with fp32 sums: codes are exact there, a query row is
 * scaled by a power of two to its largest element (elements 2^-28 below it
 * lose bits), and a token's weight times its value scale is rounded once to 11
 * bits (to fewer below 2^-21 of the row's largest); the statistics stay in
 * fp32.
 *   q  device, bf16, row r head h at q + r*ldq + h*D, 16-byte aligned, ldq a
 *      multiple of 8, at least hq*D
 *   workspace  16-byte aligned, of draft_layer_workspace_bytes() bytes
 * How the work is divided goes by the batch's averages (the results hold for any
 * batch): rows a sequence, those without rows included, choose one kernel for the
 * call, so long prompts and single tokens are faster in calls of their own (one of
 * 2,048 rows and 63 single tokens over 6,000: 225 us together, 66 and 126 apart);
 * and a batch of about 1024/hkv sequences of few rows and more (512/hkv at D =
 * 256) does not split a long context among workgroups: one of 131,072 tokens among
 * 127 of 500 and 8 kv heads takes 966 us, among 126 of them 82.
 * A row with an infinite or NaN element of q, or that sees a page whose key or
 * value scale is infinite or NaN, is NaN (out and lse), and no other row is.
 * Limits: scale finite and > 0, window >= 0, sinks >= 0.  Results hold for q
 * below 2^64 in magnitude, scales of seen pages in 2^-40 .. 2^57 and scores z_j
 * below 2^120 in magnitude (from 2^24 on fp32 holds no fractions of them).
 * Errors: DH_EINVAL, DH_ESHAPE, DH_EUNSUP, DH_EHIP.
 */
int draft_layer_attend(const void* q, int64_t ldq, const uint8_t* k_codes, const uint8_t* v_codes,
                       const float* k_scale, const float* v_scale, int n_pages, int page, const int32_t* q_start,
                       const int32_t* kv_len, const int32_t* table, int n_seq, int max_pages, int T, int hq,
                       int hkv, int D, float scale, int window, int sinks, void* out, float* lse, void* workspace,
                       size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DRAFTLAYER_H */
