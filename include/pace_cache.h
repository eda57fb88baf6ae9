/*
 * pace_cache.h -- C ABI of the attention-layer operators that serve a hybrid stack next to
 * the gated-delta layers of pace.h, for AMD Instinct MI355X (gfx950): rotary positions, a
 * paged key/value cache quantised as it is written, and attention for drafted tokens over
 * that cache (a single token and a prompt chunk are its simplest cases).
 *
 * The conventions are those of pace.h: plain C, caller-owned device memory, host-side
 * validation before any launch (PACE_EINVAL / PACE_EUNSUPPORTED, nothing touched), launch
 * errors as PACE_EHIP, no global state, no allocation and no synchronisation.  Every call
 * only enqueues kernels on `stream` (a hipStream_t, NULL = default stream) and may be
 * captured in a HIP graph.  Memory handed to a call must stay allocated, and must not be
 * written by other streams, until the call's kernels have run.
 *
 * ------------------------------------------------------------------------------------
 * Notation
 *   B sequences, T tokens of each in the call, Hq query heads, Hkv key/value heads
 *   (Hq % Hkv == 0; query head h reads key/value head h / (Hq / Hkv)), d channels a head,
 *   g channels a scale group, P tokens a page.
 *
 * I/O tensors (io_dtype fp32 or bf16): element (token n, head h, channel c) of a tensor with
 * token stride `s` (in elements, s >= heads * d) is at n * s + h * d + c; tokens of [B][T]
 * are numbered b * T + t.  The stride lets q, k and v be slices of one projection's output, or the
 * last tokens of long prompts; all tokens together may span up to 2^48 bytes.
 *
 * Quantiser of the cache: the rules of pace.h's symmetric state quantiser on the vector of one
 * (token, head), each group of g contiguous channels with its own scale:
 *   M = max|x| of the group, s = bf16 rounded toward +inf of M / L,
 *   int8 (L = 127), int4 (L = 7):  c = round-half-even(x / s) clipped to +-L, x^ = s c;
 *   fp8 (L = 448):  c = x / s rounded to the nearest e4m3 value (ties to even), x^ = s c.
 * x / s is formed in fp32, correctly rounded for scales from 2^-108 on, where exact ties of bf16 inputs
 * are exact; under that it may be a unit off, so that a value within 2^-22 of a step of a tie may go
 * either way.  So that a cache holds finite values only: a NaN is stored as 0, |x| is clamped to 2^127, and
 * a group whose scale lies under 2^-126 is stored as zeros (s = 0).
 *
 * CACHE LAYOUT: num_pages pages; page p, key/value head h is a record of
 * pace_cache_layout_info.record_bytes bytes at (p * Hkv + h) * record_bytes:
 *     key codes   P d b / 8 bytes
 *     key scales  bf16 [P/4][d/g][4]: token r, group G at ((r div 4) (d/g) + G) 4 + r mod 4
 *     value codes P d b / 8 bytes
 *     value scales, as the key scales
 * Codes lie in the order in which the matrix instructions take them, so that every load of the
 * attention kernel is 16 (or 8) bytes a lane, contiguous over the lanes.  With b bits a code,
 * LB = d b / 32, W = min(16, LB), G = c div 32:
 *   keys, in tiles of 16 tokens (16 d b / 8 bytes): channel c of token r belongs to lane
 *     a = (c mod 32) div 8 of the token, which holds LB bytes; byte x of them is at
 *     (x div W) 64 W + (16 a + r mod 16) W + x mod W.
 *     8 bits: x = 8 G + c mod 8.  4 bits: the 8 channels e = c mod 8 of a unit share the four
 *     bytes from x = 4 G (little-endian), channel e in nibble e div 2 + 4 (e mod 2).
 *   values, in quads of 4 tokens (4 d b / 8 bytes): channel c belongs to lane
 *     m = (c mod 32) div 2, which holds LB bytes; byte x is at (x div W) 16 W + m W + x mod W.
 *     8 bits: x = 4 (2 G + c mod 2) + r mod 4.  4 bits: x = 4 G + r mod 4, the even channel in
 *     the low nibble, the odd one in the high.
 * Stored fields: int8 c + 128, int4 c + 8 (as in pace.h), fp8 the e4m3 bit pattern.
 * No byte holds codes of two tokens, so different tokens may be written by different calls.
 *
 * page_table: int32 [B][max_pages] on the device; entry i of a sequence is the page of its
 * positions [i P, (i + 1) P).  An entry outside [0, num_pages) marks a page that is not there:
 * writes to it are dropped, reads of it give zeros, attention does not see its positions.
 * ------------------------------------------------------------------------------------
 */
#ifndef PACE_CACHE_H
#define PACE_CACHE_H

#include "pace.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ rotary positions */

typedef enum {
  PACE_ROPE_PLAIN = 0,   /* f_i = base^(-2 i / rd) */
  PACE_ROPE_LINEAR = 1,  /* f_i / factor */
  PACE_ROPE_NTK = 2,     /* base raised to base * factor^(rd / (rd - 2)) */
  PACE_ROPE_BLEND = 3    /* by wavelength: pairs that turn more than fast_turns times over
                            original_len keep f_i, those that turn less than slow_turns times
                            take f_i / factor, a linear ramp over the pair index between;
                            magnitude 0.1 ln(factor) + 1 */
} pace_rope_scaling;

/* Frequencies (radians per position) of a rotary embedding, in fp64.  Host only.
 * Out: freqs[rd / 2]; *magnitude: the factor on the rotated values (1 except for BLEND).
 * original_len, fast_turns and slow_turns are read for BLEND only (32 and 1 are usual turns).
 * Errors: PACE_EINVAL for a null pointer, an odd rd or rd < 2, base <= 1, factor <= 0 (BLEND:
 * < 1), original_len <= 0, fast_turns <= slow_turns, slow_turns <= 0, or an unknown scaling. */
pace_status pace_rotary_freqs(int32_t rd, double base, int32_t scaling, double factor,
                              double original_len, double fast_turns, double slow_turns,
                              double* freqs, double* magnitude);

typedef struct {
  int32_t Hq, Hk;        /* heads of q and of k (either may be 0: that tensor is not touched) */
  int32_t d;             /* channels a head; any even number up to 1024 */
  int32_t rd;            /* the first rd channels are rotated (even, 2 <= rd <= min(d, 512)) */
  int32_t interleaved;   /* 0: channel i pairs with i + rd / 2;  1: 2 i with 2 i + 1 */
  int32_t io_dtype;      /* pace_io_dtype */
} pace_rotary_cfg;

/* Rotates q [n][Hq][d] and k [n][Hk][d] by their positions: with a = position * freqs[i], m = magnitude,
 *     y_i = m (x_i cos a - x_j sin a),   y_j = m (x_j cos a + x_i sin a)
 * for the pair (i, j); channels from rd on are copied.  a is formed and reduced to its fraction of a
 * turn in fp64; the fraction, its cosine and sine and their products with m are fp32.  The outputs are
 * rounded once, to the io type.
 * inverse != 0 turns by -a.  With the same m that is the transpose, which takes gradients back; its
 * inverse, which takes keys back, is the call with 1 / m.
 * positions int32 [n] (any sign), freqs fp64 [rd / 2], both on the device.  A tensor may be
 * rotated in place (output == input with the same stride); other overlaps are not allowed.
 * Pointers must be aligned to their element (16 bytes with strides of 16 bytes run fastest).
 * n == 0 is allowed and does nothing.
 * Errors: PACE_EINVAL for null pointers, bad sizes or strides, misalignment, a magnitude that is not
 * finite in fp32; PACE_EUNSUPPORTED for d or rd outside the range above. */
pace_status pace_rotary(const pace_rotary_cfg* cfg, int32_t n, const int32_t* positions,
                        const double* freqs, double magnitude, int32_t inverse, const void* q,
                        int64_t q_stride, const void* k, int64_t k_stride, void* q_out,
                        int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream);

/* ------------------------------------------------------------------- the cache itself */

typedef enum { PACE_CACHE_INT8 = 0, PACE_CACHE_INT4 = 1, PACE_CACHE_FP8 = 2 } pace_cache_kind;

/* Supported by the kernels: d in {64, 128, 256}; group in {32, 64, 128} with group | d; page a
 * power of two in [16, 1024]; Hq % Hkv == 0, Hq <= 1024; 1 <= B <= 65535;
 * max_pages * page < 2^31. */
typedef struct {
  int32_t B, Hq, Hkv, d;
  int32_t kind;          /* pace_cache_kind */
  int32_t group;         /* channels a scale */
  int32_t page;          /* tokens a page */
  int32_t num_pages;     /* pages of the pool */
  int32_t max_pages;     /* page_table entries a sequence */
  int32_t io_dtype;      /* pace_io_dtype of q, k, v, o */
} pace_cache_cfg;

typedef struct {
  size_t cache_bytes;    /* the whole pool */
  size_t page_bytes;     /* one page, all heads */
  size_t record_bytes;   /* one page of one head */
  double bits_per_value; /* codes and scales: b + 16 / g */
} pace_cache_layout_info;

/* Sizes of a cache.  Host only.  Errors as for every call with this configuration: PACE_EINVAL
 * malformed, PACE_EUNSUPPORTED outside the kernels' range. */
pace_status pace_cache_layout(const pace_cache_cfg* cfg, pace_cache_layout_info* out);

/* Quantises k, v [B][T][Hkv][d] and stores them at positions int32 [B][T] (device) of their
 * sequences.  A negative position, one past max_pages * P, or one whose page is not there is
 * skipped; the positions of one sequence must differ.  Runs of consecutive positions are
 * stored fastest.  cache must be 256-byte aligned, k and v 16-byte (strides too).
 * T == 0 is allowed and does nothing.
 * PACE_EUNSUPPORTED where B Hkv ceil((T + 15) / 16) (T < 16: B Hkv) is over 2^26 - 4; reading, too. */
pace_status pace_cache_write(const pace_cache_cfg* cfg, void* cache, const int32_t* page_table,
                             const int32_t* positions, int32_t T, const void* k, int64_t k_stride,
                             const void* v, int64_t v_stride, void* stream);

/* The reverse: k, v [B][T][Hkv][d] from positions int32 [B][T] (device), each value s c rounded
 * once to the io type; zeros where a position is skipped. */
pace_status pace_cache_read(const pace_cache_cfg* cfg, const void* cache,
                            const int32_t* page_table, const int32_t* positions, int32_t T,
                            void* k, int64_t k_stride, void* v, int64_t v_stride, void* stream);

/* ------------------------------------------------------- attention for drafted tokens */

/* Ancestor bits of trees of drafted tokens.  Host only.  parents[T]: the node that token i
 * hangs on, or -1 for the sequence itself; parents[i] < i.  bits: T rows of
 * ceil(T / 32) words; bit j of row i says that token j is i or one of its ancestors.
 * Errors: PACE_EINVAL for null pointers, T < 1 or a parent outside [-1, i). */
pace_status pace_tree_bits(const int32_t* parents, int32_t T, uint32_t* bits);

/* o = softmax(scale q k^T) v for T tokens of each sequence, whose keys and values were written
 * to the cache at positions ctx_lens[b] .. ctx_lens[b] + T - 1 before.  Token i of sequence b
 * sees every position below ctx_lens[b], and position ctx_lens[b] + j if
 *     tree == NULL:  j <= i   (a single token, a prompt chunk, a chain of drafts)
 *     else:          bit j of its row, tree[b * tree_stride + i * ceil(T / 32) + j / 32]
 * (uint32 words on the device; tree_stride in words, 0: one tree for all sequences).
 * draft_lens int32 [B] (device, may be NULL = T): sequence b has only draft_lens[b] tokens;
 * later rows see nothing, later positions are seen by nobody.
 * A row that sees nothing gets o = 0, lse = -inf.  What lies in the cache beyond the
 * sequences' ends is never used, whatever its bytes.
 * q [B][T][Hq][d] (token stride q_stride, 16-byte aligned), o [B][T][Hq][d] contiguous,
 * lse fp32 [B][T][Hq] (may be NULL): ln sum exp(scale q k).  ctx_lens int32 [B] (device),
 * negative = 0.
 * Computed with matrix instructions on exact codes: fp16 operands with fp32 accumulation for
 * bf16 I/O, two-piece operands (22 bits) for fp32 I/O; softmax statistics and outputs are kept in fp32 and
 * rounded once.  Weights, times their value scales, are rounded to 11 (22) bits in a unit of their row and
 * channel group; one under 2^-17 (fp32: 2^-5) of the row's largest such product keeps fewer of them, and is
 * off by at most 2^-28 of that product.  What a row does not see has no part in it.
 * Scores are right as long as they, and their parts of a group of channels, fit fp32 in base 2 (2.3e38); a
 * key may hold 2^127.  A query that is not finite makes its own row NaN, and no other.
 * For one B, T and max_len a result repeats bit for bit and does not depend on the other sequences' lengths
 * and contents; another B or max_len may cut a context otherwise, which changes the order of its sums.
 * max_len: upper bound of ctx_lens[b] + T that the work is laid out for (host); a longer
 * sequence is still computed in full, only less evenly spread.
 * workspace: pace_cache_attention_workspace_bytes(cfg, T, max_len) bytes, 256-byte aligned
 * (NULL if 0).
 * Errors: PACE_EINVAL for null pointers, T < 1, max_len < 1, a negative tree_stride, a
 * scale over 2.3e38 in magnitude or not finite, a workspace that is too small, misalignment; PACE_EUNSUPPORTED for
 * T * Hq / Hkv over 2^24, 2^31 rows (B T Hq) in all or more, or 2^24 workgroups or more (one for every 16
 * or 32 rows of a sequence and key/value head, times the pieces of a context where there are few). */
pace_status pace_cache_attention(const pace_cache_cfg* cfg, const void* cache,
                                 const int32_t* page_table, const void* q, int64_t q_stride,
                                 int32_t T, const int32_t* ctx_lens, const int32_t* draft_lens,
                                 const uint32_t* tree, int64_t tree_stride, double scale,
                                 int32_t max_len, void* o, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* Workspace bytes of pace_cache_attention, written to *bytes_out (0: none needed).  Host only.
 * Errors (nothing is written) as pace_cache_attention. */
pace_status pace_cache_attention_workspace_bytes(const pace_cache_cfg* cfg, int32_t T,
                                                 int32_t max_len, size_t* bytes_out);

#ifdef __cplusplus
}
#endif
#endif /* PACE_CACHE_H */
