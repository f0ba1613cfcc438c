/*
 * qsa_cache.h -- bounded caches for long decodes: K/V rows held in 8 or 4 bits, the
 * attention that reads them, and the eviction of groups by the attention that
 * they have received.  Part of libqsa; the conventions of qsa.h hold for every
 * call here (device pointers of the current device, the caller owns every
 * buffer, asynchronous on `stream`, host-detectable errors before anything is
 * enqueued, device-detected errors in the workspace's sticky error word,
 * results that depend neither on the rest of the batch nor on the number of
 * SMs, calls that share a workspace must not overlap on the GPU).  Kernels are
 * launched programmatically, as qsa_score_pooled's is: each waits for the kernel
 * before it on `stream` before it reads or writes anything, so stream order holds.
 *
 * The notes that define the method have no counterpart to this header.  It
 * keeps to their units: the four-token group that is scored, selected and
 * gathered whole ([AFN-017] Decision) is the block that shares a scale and the
 * unit that is evicted, and the raw tail of at most 3 tokens stays in the f32
 * K/V cache until its group completes, as it stays unscored until then.
 */
#ifndef QSA_CACHE_H
#define QSA_CACHE_H

#include "qsa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- the coded cache ------------------------------------------------------ */

#define QSA_CODE_E4M3 0 /* 8-bit float, 4 exponent and 3 mantissa bits, largest value 448 */
#define QSA_CODE_INT8 1 /* signed integer, -127 .. 127                                    */
#define QSA_CODE_E2M1 4 /* 4-bit float, 2 exponent and 1 mantissa bits: 0, 0.5, 1, 1.5, 2, 3, 4, 6, and negative */
#define QSA_CODE_INT4 5 /* 4-bit integer, -7 .. 7, stored as 1 .. 15                      */

/* K and V of complete groups, one block per group, by PHYSICAL block number.
 * A code c of K in block p and KV head h stands for scales[p][h][0] * c, one
 * of V for scales[p][h][1] * c.  Layout of a (block, head), 8*d bytes:
 *   K: [d/64][4 tokens][64 dims]    code of token u, dim j at (j/64)*256 + u*64 + j%64
 *   V: [d][4 tokens]                code of token u, dim j at 4*d + 4*j + u
 * (K: the 16 codes that one lane of the attention's matrix product holds sit
 * side by side and two tokens fill the 128 bytes that shared memory serves at
 * once; V: the four tokens of one dim are the operand word of the second
 * product).  A scale is finite, or NaN for a group that held a value that is
 * not finite: every output that attends to such a group is NaN.
 *
 * In 4 bits each tile of four tokens by four neighbouring dims (4r .. 4r+3) has a scale
 * of its own besides, an e4m3 number t >= 0, and a code c stands for scales[p][h][.] * t * c:
 * 4.5 bits a value.  Layout of a (block, head), 9*d/2 bytes; a word is 32 bits, least
 * significant byte first, and holds four pairs of codes p = 0 .. 3 -- for e2m1 in the low and
 * the high half of byte p, for int4 in bits 4p .. 4p+3 and 4p+16 .. 4p+19, as code + 8:
 *   K: [d/64 j][2 i][4 c][2 t][2 w] words at byte 128*j + 64*i + 16*c + 8*t + 4*w: pair p of
 *      token 2t + i is dims 64j + 16c + 8w + p and + 4
 *   V: [d/64 m][8 h][2 n][2 w] words at byte 2*d + 128*m + 16*h + 8*n + 4*w: pair p of dim
 *      64m + 32n + 4h + 2w + p/2 is tokens 2(p%2) and + 1
 *   tile scales of K at byte 4*d: that of dims 64j + 16c + 4r .. at c*d/16 + 4j + r
 *   tile scales of V at byte 4*d + d/4: that of dims 64m + 32n + 4h .. at h*d/32 + 2m + n
 * (what a lane of the attention's products holds sits side by side, and the two codes of a
 * pair are the two halves of one of its operand registers). */
typedef struct {
    uint8_t *codes;              /* [num_blocks, n_kv, 8*d], or 9*d/2 in 4 bits; 16-byte aligned */
    float *scales;               /* [num_blocks, n_kv, 2], 16-byte aligned                 */
    int64_t num_blocks;
    const int32_t *block_map;    /* logical -> physical: group g of query b is in block    */
                                 /*   block_map[block_offset[b] + g]                       */
    const int64_t *block_offset; /* [B] first block-map entry of query b's history         */
    int32_t format;              /* QSA_CODE_E4M3, _INT8, _E2M1 or _INT4                   */
} qsa_coded_cache;

/* Codes complete groups: for each query b and g in [group_begin[b],
 * group_end[b]) (device int32 arrays), the f32 rows of tokens 4g..4g+3 --
 * k_cache / v_cache rows slot_map[slot_offset[b] + 4g + u], read from `in`,
 * whose other members may be NULL -- are coded into block
 * block_map[block_offset[b] + g], per KV head and for K and V apart:
 *   s = max |x| * r  (r = 1/448 for e4m3, 1/127 for int8, rounded to binary32;
 *   over 4 tokens x d),   code = round_to_nearest_even(x / s),
 * product and quotient binary32, correctly rounded (an e4m3 code of a negative
 * value that rounds to zero, or of -0, is -0: 0x80).  A scale below the smallest
 * normal float is stored as 0 with codes 0 (the group is flushed to zero); a
 * group with a value that is not finite gets the scale NaN and codes 0.
 * In 4 bits, with c = 6 (e2m1) or 7 (int4), per KV head and for K and V apart:
 *   s = max |x| * rn(1 / (448 c)) over 4 tokens x d, flushed as above (then with tile scales 0);
 *   t = e4m3(min(448, a / (c s))) of each tile, a = max |x| over its 16 values;
 *   code = round_to_nearest_even(x / (t s)), at most c in size, or 0 where t = 0,
 * every product and quotient binary32, correctly rounded, t to the nearest e4m3 number (even
 * on ties; a tile below about 2^-19 of the group's largest value gets 0), codes to the nearest
 * number of their format (the one with an even last bit on ties).
 * Afterwards nothing here reads those f32 rows again: their slots may be
 * reused (a later tail's, for instance).  max_groups (host) bounds group_end[b]
 * - group_begin[b] for every b and sizes the launch: a decode step that
 * completes one group per query passes 1.  Two queries may name the same block
 * only with the same rows.  A range outside [0, max_visible/4] or longer than
 * max_groups is skipped (QSA_DEVERR_VISIBLE_RANGE); a block outside
 * [0, num_blocks) is skipped and a row outside [0, num_slots) is taken as zeros
 * (both QSA_DEVERR_SLOT_RANGE).  Workspace: qsa_workspace_size(dims). */
qsa_status qsa_code_groups(const qsa_dims *dims, const qsa_inputs *in, const qsa_coded_cache *cache,
                           const int32_t *group_begin, const int32_t *group_end, int32_t max_groups,
                           void *ws, size_t ws_bytes, void *stream);

/* Workspace of the calls below that attend over a coded cache (0 if the dims
 * are invalid): qsa_workspace_size(dims) when both flags are 0, followed by
 *   whole_history: the attention's partial states, n_q*(d+2) floats per run of
 *     a row and query, at most 513 runs;
 *   with_weights: n_q * (1.25 * groups of a row + 2) + 2 floats per query, groups =
 *     max_visible/4 for whole histories, else budget_groups.
 * Linear in the history, never queries x keys of other queries.  A workspace
 * made for both flags serves every call of this library with these dims. */
size_t qsa_coded_workspace_size(const qsa_dims *dims, int32_t whole_history, int32_t with_weights);

/* Attention over the coded cache.  For each query b and head h (KV head
 * h / (n_q/n_kv)), over the row's tokens t:
 *   x_t = scale * q[b][h] . k_t,   out[b][h] = sum_t softmax(x)_t v_t.
 * The row:
 *   ids, n_ids given: the tokens ids[b*row_cap + i], i < n_ids[b], laid out as
 *     qsa_select emits them -- complete groups (four consecutive IDs from a
 *     multiple of 4), then n_ids[b] mod 4 single tokens;
 *   ids = n_ids = NULL: every visible token, 0 .. visible[b]-1 (up to
 *     QSA_MAX_VISIBLE).
 * Groups are read from the coded cache, the last (row length mod 4) tokens
 * from the f32 k_cache / v_cache through the slot map.  An empty row gives a
 * zero output, and so does a head whose scores are all -inf (below binary32's
 * range), which adds no weight either.  Reads in->q, visible, slot_map,
 * slot_offset, k_cache, v_cache.  out: [B, n_q, d].
 *
 * weights (NULL: none): accumulated attention.  weights[weight_offset[b] + g]
 * += sum over heads h and over the row's tokens t of group g = t/4 of
 * softmax(x)_t, the incomplete last group (g = visible[b]/4) included, so one
 * query adds n_q in all; a row with a score that is NaN makes its groups' weights
 * NaN.  Shares are added to what is there: the caller sets a group's entry to 0
 * when its first token comes.  Queries with the same weight_offset share a history:
 * their shares are added in a fixed order, so the sum has one value (the rows of
 * different offsets must not overlap).
 *
 * The codes, in 4 bits times their tile scales, are exact in 16-bit floats; q and the softmax weights (each times its
 * group's V scale, in binary32) enter the products as a sum of two 16-bit floats:
 * to 2^-22 of themselves, or 2^-37 of the largest of the head's q, of the head's
 * weights in four (in 4 bits: eight) consecutive groups of the row, where that is more.  All sums,
 * maxima and outputs are binary32.  Three products have to stay below 2^128 for
 * that: scale times a head's largest |q| times a K scale, and, as a weight is up to
 * 2^8 before the division by their sum, 2^8 times the sum of a row's |v| and 2^8 times
 * a V scale (which the one before it implies for groups that qsa_code_groups coded).
 * Where a head's q is not all zeros, its largest |q| is at least 2^-110, and scale
 * times that at least 2^-112.
 *
 * A count outside [0, row_cap] or a T_b outside [0, max_visible] gives a zero
 * output (QSA_DEVERR_ROW_RANGE / QSA_DEVERR_VISIBLE_RANGE) and adds no weight;
 * an ID outside [0, visible[b]) or out of the layout above, a block outside
 * [0, num_blocks) and a slot outside [0, num_slots) are taken as zero K/V rows
 * and flagged (QSA_DEVERR_ROW_RANGE / QSA_DEVERR_SLOT_RANGE).  With weights,
 * a query whose row has IDs out of that layout, or groups that do not ascend,
 * adds no weight (QSA_DEVERR_ROW_RANGE).
 * Workspace: qsa_coded_workspace_size(dims, ids == NULL, weights != NULL). */
qsa_status qsa_attend_coded(const qsa_dims *dims, const qsa_inputs *in, const qsa_coded_cache *cache,
                            const int32_t *ids, const int32_t *n_ids, float *out, float *weights,
                            const int64_t *weight_offset, void *ws, size_t ws_bytes, void *stream);

/* The whole path with a coded cache: scores (from the pooled-key cache when
 * pooled is given, as qsa_decode_pooled, else from the raw index keys, as
 * qsa_decode), qsa_select, then qsa_attend_coded over the chosen rows.  ids,
 * n_ids: bit-identical to qsa_decode's; out and weights as qsa_attend_coded.
 * ids, n_ids and out may point to mapped (pinned) host memory.
 * Workspace: qsa_coded_workspace_size(dims, 0, weights != NULL). */
qsa_status qsa_decode_coded(const qsa_dims *dims, const qsa_inputs *in, const qsa_coded_cache *cache,
                            const float *pooled, const int64_t *pool_offset, int32_t *ids, int32_t *n_ids,
                            float *out, float *weights, const int64_t *weight_offset, void *ws,
                            size_t ws_bytes, void *stream);

/* ---- eviction -------------------------------------------------------------- */

/* The groups each history keeps.  With G = visible[b]/4 complete groups and
 * weights[weight_offset[b] + g], keeps min(G, keep_groups) of them: all if
 * G <= keep_groups, else the first sink_groups, the last recent_groups and,
 * among the others, the best by (weight descending, group position ascending)
 * -- ties resolved while choosing membership, as in qsa_select; a NaN weight
 * ranks below every number.  kept: [B, keep_groups] int32, ascending positions,
 * entries >= n_kept[b] untouched; n_kept: [B].  evicted (NULL: not wanted):
 * [B, max_visible/4] int32, the other groups in ascending order, entries >= G
 * - n_kept[b] untouched: what the caller gives back to its allocators.
 * 1 <= keep_groups <= QSA_MAX_VISIBLE/4, 0 <= sink_groups, recent_groups,
 * sink_groups + recent_groups <= keep_groups.  A T_b outside [0, max_visible]
 * keeps nothing (QSA_DEVERR_VISIBLE_RANGE).
 * Workspace: qsa_workspace_size(dims). */
qsa_status qsa_evict_select(const qsa_dims *dims, const int32_t *visible, const float *weights,
                            const int64_t *weight_offset, int32_t keep_groups, int32_t sink_groups,
                            int32_t recent_groups, int32_t *kept, int32_t *n_kept, int32_t *evicted,
                            void *ws, size_t ws_bytes, void *stream);

/* What describes a batch of histories in logical order: the arrays that the
 * other calls read, each with the first row of query b's history.  A member
 * that is NULL in both histories of a call (and its offsets) is not moved. */
typedef struct {
    float *idx_keys;             /* raw index keys, one row of d_I floats per token     */
    const int64_t *key_offset;
    float *pooled;               /* pooled keys, one row of d_I floats per group        */
    const int64_t *pool_offset;
    int32_t *slot_map;           /* one entry per token                                 */
    const int64_t *slot_offset;
    int32_t *block_map;          /* one entry per group                                 */
    const int64_t *block_offset;
    float *weights;              /* one entry per group, and one for an incomplete one  */
    const int64_t *weight_offset;
    int32_t *visible;            /* [B] T_b                                             */
} qsa_history;

/* Moves the kept groups of `src` to `dst`, where group kept[b][i] becomes group
 * i, with the raw tail behind them, and sets dst->visible[b] = 4*n_kept[b] +
 * T_b mod 4: raw index keys, pooled keys (in the layout of their new position),
 * slot map, block map and accumulated weights (of an incomplete last group too;
 * with T_b mod 4 == 0 entry n_kept[b] is behind the region's end, and the caller's
 * to set to 0 when the next group starts).  The K/V rows and codes do not move: the
 * maps follow them.  kept, n_kept: as qsa_evict_select fills them,
 * [B, keep_groups] and [B].  dst's regions hold 4*n_kept[b] + 3 tokens or what
 * the caller knows to be enough, overlap neither each other nor src's; rows
 * behind a region's new end are left as they were.  src->visible and
 * dst->visible are required.  A count outside [0, min(keep_groups, T_b/4)], or
 * T_b outside [0, max_visible], leaves that history out with dst->visible[b] =
 * 0; a position outside [0, T_b/4) zero-fills its rows and sets its maps' new
 * entries to -1 (all QSA_DEVERR_ROW_RANGE / QSA_DEVERR_VISIBLE_RANGE).  d_I is
 * 32 or 64.  Workspace: qsa_workspace_size(dims). */
qsa_status qsa_evict_compact(const qsa_dims *dims, int32_t keep_groups, const int32_t *kept,
                             const int32_t *n_kept, const qsa_history *src, const qsa_history *dst, void *ws,
                             size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QSA_CACHE_H */
