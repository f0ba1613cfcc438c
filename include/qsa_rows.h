/*
 * qsa_rows.h -- K/V rows on their way into the caches and back: a new token's
 * projections normalised, rotated and written where the path reads them, and
 * coded groups read back as f32 rows.  Part of libqsa; the conventions of
 * qsa.h hold for every call here (device pointers of the current device, the
 * caller owns every buffer, asynchronous on `stream`, host-detectable errors
 * before anything is enqueued, device-detected errors in the workspace's sticky
 * error word, results that do not depend on the rest of the batch).  Kernels are
 * launched programmatically, as those of qsa_cache.h: each waits for the kernel
 * before it on `stream` before it reads or writes anything, so stream order holds.
 *
 * The notes that define the method start from finished queries, index keys and
 * K/V rows and have no counterpart to this header.
 */
#ifndef QSA_ROWS_H
#define QSA_ROWS_H

#include "qsa_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The calls here use the error word at a workspace's start and nothing else of it: a
 * zeroed workspace of this size serves them, whatever the dims, and so does any that
 * serves other calls. */
#define QSA_ROWS_WORKSPACE_BYTES 256

/* ---- new tokens -------------------------------------------------------------- */

/* Element types of projected rows. */
#define QSA_ROWS_F32 0
#define QSA_ROWS_BF16 1
#define QSA_ROWS_F16 2

/* Which dims of a head are rotated together, of its first `dims`. */
#define QSA_PAIR_HALVES 0      /* j and j + dims/2  */
#define QSA_PAIR_NEIGHBOURS 1  /* 2j and 2j + 1     */

#define QSA_MAX_AXES 4

/* One projection of the batch's new tokens.  The row of query b starts at element
 * b*stride of `rows` and holds its heads side by side.  Rows overlap nothing that the call
 * writes, but f32 rows of q or q_idx may be in->q or in->q_idx themselves, one query's behind
 * the other's as there (stride heads*width).  `rows` NULL: this projection is not given, and
 * what it would write stays as it is. */
typedef struct {
    const void *rows;            /* 16-byte aligned                                             */
    int64_t stride;              /* elements; at least heads*width, and 16 bytes' worth a multiple */
    const float *norm;           /* [width], 16-byte aligned: the weights of each head's norm; NULL: none */
} qsa_projection;

/* The rotation of one width of heads: pair j of `pairing` turns by the angle
 *   sum over axes a of positions[a][b] * freq[a][j].  */
typedef struct {
    const float *freq;           /* [axes, dims/2], 4-byte aligned: radians per step of each axis, finite
                                    and below 2^16 in size; 0 where an axis does not turn a pair    */
    int32_t dims;                /* rotated dims, the first of each head: a multiple of 8 up to the width; 0: none */
    int32_t pairing;             /* QSA_PAIR_HALVES or QSA_PAIR_NEIGHBOURS                       */
} qsa_rotation;

typedef struct {
    qsa_projection q, k, v;      /* n_q, n_kv and n_kv heads of d (v: no norm)                   */
    qsa_projection q_idx;        /* H_I heads of d_I                                             */
    qsa_projection idx_key;      /* one head of d_I                                              */
    int32_t type;                /* QSA_ROWS_*, of every projection                              */
    int32_t axes;                /* 1 .. QSA_MAX_AXES                                            */
    const int32_t *positions;    /* [axes, B]: the new token of query b; any value (they need not
                                    be its place in the history, which an eviction changes); may be
                                    NULL if nothing is rotated                                   */
    qsa_rotation turn;           /* of q and k                                                   */
    qsa_rotation turn_idx;       /* of q_idx and idx_key                                         */
    float eps;                   /* of the norms, >= 0                                           */
} qsa_new_tokens;

/* Writes the new token of every query -- the last of its visible[b] tokens, t =
 * visible[b] - 1 -- where the other calls read it.  Per head x of a projection:
 *   y = x * w / sqrt(mean(x^2) + eps)   (w = norm; y = x where that is NULL),
 *   (z_i, z_k) = (y_i cos - y_k sin, y_i sin + y_k cos)  for its rotated pairs (i, k),
 * and z, in binary32, goes to
 *   q:       in->q[b]                q_idx:  in->q_idx[b]
 *   idx_key: in->idx_keys row key_offset[b] + t
 *   k, v:    in->k_cache / v_cache row slot_map[slot_offset[b] + t]   (v as it is)
 * which are written through the pointers of `in`, whose const stands for the other calls.
 * A decode step passes one query per sequence, a chunked prefill its consecutive
 * positions of one history; then the group that a token completes can be pooled
 * (qsa_pool_groups) and coded (qsa_code_groups).  Reads in->visible, and slot_map,
 * slot_offset or key_offset where a projection goes there; the members of `in` that no
 * given projection needs may be NULL.  No two queries may name the same place.
 *
 * Everything after the load is binary32; the angle is kept as a fraction of a full turn
 * to (axes + 3) * 2^-34 whatever the position, so far positions lose nothing, and its sine and
 * cosine are off by at most 2^-22.  The sum of a head's squares has to stay below 2^128; it may be
 * as small as it likes, but for a head of zeros, which with eps = 0 is NaN.  A frequency that
 * is not finite or not below 2^16 in size makes its pair NaN.
 * T_b = 0: the query has no new token, and nothing of it is written.  A T_b outside
 * [0, max_visible] gives zero rows in in->q and in->q_idx and no other
 * (QSA_DEVERR_VISIBLE_RANGE), a slot outside [0, num_slots) no K/V row
 * (QSA_DEVERR_SLOT_RANGE).
 * Refused (QSA_ERR_INVALID_ARG): no projection at all, a stride or an alignment other
 * than the above, v.norm, a rotation with `dims` that is not a multiple of 8 or wider than
 * the head, without frequencies or positions, rows that start where they are written to (but the
 * f32 queries above); QSA_ERR_UNSUPPORTED_SHAPE: d not 64 or 128
 * with q, k or v given, d_I not 32 or 64 with q_idx or idx_key given.
 * Workspace: QSA_ROWS_WORKSPACE_BYTES. */
qsa_status qsa_append_tokens(const qsa_dims *dims, const qsa_inputs *in, const qsa_new_tokens *tokens,
                             void *ws, size_t ws_bytes, void *stream);

/* ---- coded groups read back --------------------------------------------------- */

/* The way back of qsa_code_groups, for every format: for each query b and g in
 * [group_begin[b], group_end[b]) (device int32 arrays), the values that block
 * block_map[block_offset[b] + g] stands for -- the product of a code (in 4 bits times its
 * tile scale, which is exact) and its scale, rounded to binary32 once -- go to the f32 rows of tokens
 * 4g..4g+3, in->k_cache / v_cache rows slot_map[slot_offset[b] + 4g + u], which are written
 * through the pointers of `in`.  For histories that go on in f32 or in another format, or
 * leave the device.  max_groups bounds every range as in qsa_code_groups; two queries may
 * name the same slot only with the same block.  A range outside [0, max_visible/4] or
 * longer than max_groups is skipped (QSA_DEVERR_VISIBLE_RANGE); a block outside
 * [0, num_blocks) gives zero rows, a slot outside [0, num_slots) is skipped (both
 * QSA_DEVERR_SLOT_RANGE).  Reads no other member of `in`.  Workspace: QSA_ROWS_WORKSPACE_BYTES. */
qsa_status qsa_read_groups(const qsa_dims *dims, const qsa_inputs *in, const qsa_coded_cache *cache,
                           const int32_t *group_begin, const int32_t *group_end, int32_t max_groups,
                           void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QSA_ROWS_H */
