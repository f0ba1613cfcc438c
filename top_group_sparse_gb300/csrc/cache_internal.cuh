// cache_internal.cuh -- internal declarations of the coded cache, the attention
// over it and the eviction (include/qsa_cache.h), and of the rows on their way into
// the caches and back (include/qsa_rows.h).
#pragma once

#include "qsa_cache.h"
#include "qsa_internal.cuh"
#include "qsa_rows.h"

namespace qsa {

// ---- how a row is cut ---------------------------------------------------------
// A row of n complete groups is cut into runs of coded_run_groups(n) consecutive
// groups, one CTA per (run, KV head, query), and its raw tail is one more run, the
// last.  The cut depends on the row's own length and on the heads per KV
// head only, so the bits of an output do not depend on the batch.  Shorter runs
// spread a row over more SMs, longer ones pay less for a CTA's start and for the
// partial states (n_q/n_kv * (d+2) * 4 bytes per run against 8*d per group).
// Measured (this kernel alone, us): 64 rows of 1,024 groups, 8 heads of their own x
// 64: runs of 32 84, of 64 63, of 128 55; one such row 4.2, 4.8, 6.7.  64 rows of 4,096
// groups, 16 / 2 heads x 128: runs of 64 107, of 128 96; 32 ragged rows of up to
// 16,384 groups: runs of 128 95, of 256 84.  4 rows of 10,000 groups with 16 heads on
// one: 128 19, 256 27.  Selected rows (at most 512 groups): 128 queries 45, 35, 31 with
// runs of 32, 64, 128; 8 queries 5.1, 5.3, 7.2.  Beyond 131,072 groups (65,536 with 9
// to 16 heads per KV head, whose runs are half as long) the length doubles so that a
// row has at most 512 runs.
constexpr int kCodedRunRows = 64;

__host__ __device__ inline int coded_run_groups(int groups, bool whole, int heads_per_kv)
{
    if (!whole) return kCodedRunRows;
    if (groups <= 1024) return 64;
    if (groups <= 4096) return 128;
    int r = heads_per_kv > 8 ? 128 : 256;
    while ((groups + r - 1) / r > 512) r *= 2;
    return r;
}

// Upper bound of the runs (the tail's not included) of any row of at most max_groups complete groups.
inline int coded_max_runs(int max_groups, bool whole, int heads_per_kv)
{
    auto runs = [&](int g) {
        const int r = coded_run_groups(g, whole, heads_per_kv);
        return (g + r - 1) / r;
    };
    int n = runs(max_groups);
    if (whole) {  // the counts at the ends of the ranges that share a run length
        for (int edge = 1024; edge < max_groups; edge *= 2) n = n > runs(edge) ? n : runs(edge);
    }
    return n;
}

__host__ __device__ inline int coded_runs(int groups, bool whole, int heads_per_kv)
{
    const int per = coded_run_groups(groups, whole, heads_per_kv);
    return (groups + per - 1) / per;
}

struct CodedLayout {
    Layout base;
    int nparts;           // partial states per (query, head): the runs and the tail
    int mass_stride;      // group shares per (query, head); a multiple of 4
    size_t off_part_m, off_part_l, off_part_acc;  // [B, n_q, nparts], acc with d floats each
    size_t off_mass;      // [B, n_q, mass_stride]: sum of e^(x - mref) of each group
    size_t off_mref;      // [B, n_q, mass_stride/4]: the reference of four groups
    size_t off_stat;      // [B, n_q, 2]: the row's maximum and 1/denominator
    size_t off_sharing;   // [B]: whether the row may add weights, and to accumulators of its own
    size_t off_tail;      // [B]: the raw tail's share, where accumulators are shared
    int map_stride;       // selected rows: [B, map_stride] shares by group, in the scores' place
    size_t total;
};
CodedLayout make_coded_layout(const qsa_dims *d, bool whole, bool weights);

struct CodeArgs {
    const float *k_cache, *v_cache;
    int64_t num_slots;
    const int32_t *slot_map;
    const int64_t *slot_offset;
    const int32_t *group_begin, *group_end;
    uint8_t *codes;
    float *scales;
    int64_t num_blocks;
    const int32_t *block_map;
    const int64_t *block_offset;
    int32_t format, batch, kv_heads, head_dim, max_groups, g_max;
    uint32_t *err;
};
cudaError_t launch_code_groups(const CodeArgs &a, cudaStream_t s);
// The way back: codes and scales are read, k_cache and v_cache written.
cudaError_t launch_read_groups(const CodeArgs &a, cudaStream_t s);

// Bytes of one (group, KV head)'s codes; in 4 bits with their tile scales.
__host__ __device__ constexpr bool is_4bit(int format) { return format == QSA_CODE_E2M1 || format == QSA_CODE_INT4; }
__host__ __device__ constexpr int code_bytes(int format, int d) { return is_4bit(format) ? 9 * d / 2 : 8 * d; }
inline bool format_known(int f)
{
    return f == QSA_CODE_E4M3 || f == QSA_CODE_INT8 || f == QSA_CODE_E2M1 || f == QSA_CODE_INT4;
}

// Heads of one width that a new token brings: q, k and v, or q_idx and idx_key.
struct AppendFamily {
    const void *rows[3];
    int64_t stride[3];
    const float *norm[3];
    float *out[3];          // [0]: a row per query; the others: by slot, or by logical row
    int32_t heads[3];       // 0: not given
    int32_t dims, neighbours;
    const float *freq;
    int32_t wide;                  // the launcher's: every out is 32-byte aligned
    int32_t kind_steps[3], steps;  // the launcher's: a step is 256/width heads of a projection
};
struct AppendArgs {
    AppendFamily family[2];
    const int32_t *positions, *visible, *slot_map;
    const int64_t *slot_offset, *key_offset;
    int64_t num_slots;
    float eps;
    int32_t axes, batch, max_visible;
    int32_t tokens;         // the launcher's: of a CTA at a time
    uint32_t *err;
};
cudaError_t launch_append(AppendArgs a, int type, int head_dim, int idx_dim, int num_sms, cudaStream_t s);

struct AttendCodedArgs {
    const float *q;
    const int32_t *visible;
    const int32_t *ids, *n_ids;     // nullptr: whole histories
    int32_t *ids_out, *n_ids_out;   // the caller's copy of the rows (nullptr: not wanted)
    const uint8_t *codes;
    const float *scales;
    int64_t num_blocks;
    const int32_t *block_map;
    const int64_t *block_offset;
    const float *k_cache, *v_cache;
    int64_t num_slots;
    const int32_t *slot_map;
    const int64_t *slot_offset;
    float *out;
    float *part_m, *part_l, *part_acc;
    float *mass, *mref, *stat;      // nullptr: no weights
    uint32_t *sharing;
    float *share_map, *tail_share;
    float *weights;
    const int64_t *weight_offset;
    int32_t format, batch, q_heads, kv_heads, head_dim, row_cap, nparts, mass_stride, map_stride, max_visible;
    float scale;
    uint32_t *err;
};
bool attend_coded_shape_supported(int head_dim, int q_heads, int kv_heads);
cudaError_t launch_merge_coded(const AttendCodedArgs &a, cudaStream_t s);  // after the runs' states
cudaError_t launch_attend_coded(const AttendCodedArgs &a, cudaStream_t s);
cudaError_t launch_attend_coded4(const AttendCodedArgs &a, int runs, cudaStream_t s);  // the runs alone, 4-bit formats

struct EvictSelectArgs {
    const int32_t *visible;
    const float *weights;
    const int64_t *weight_offset;
    int32_t *kept, *n_kept, *evicted;
    int32_t batch, max_visible, keep, sink, recent;
    uint32_t *err;
};
cudaError_t launch_evict_select(const EvictSelectArgs &a, cudaStream_t s);

struct EvictCompactArgs {
    const int32_t *kept, *n_kept;
    qsa_history src, dst;
    int32_t batch, max_visible, keep, idx_dim;
    uint32_t *err;
};
cudaError_t launch_evict_compact(const EvictCompactArgs &a, int num_sms, cudaStream_t s);

// api.cu: qsa_score_groups / qsa_score_pooled and qsa_select as qsa_decode runs
// them (rows and counts to the workspace, selection hints, overlapped launches).
qsa_status score_and_select(const qsa_dims *d, const qsa_inputs *in, const float *pooled, const int64_t *pool_offset,
                            void *ws, const Layout &L, cudaStream_t s);
int num_sms_of_current_device();
// api_cache.cu: the f32 cache behind the slot map, and a coded cache, as arguments.
qsa_status check_rows(const qsa_inputs *in);
qsa_status check_cache(const qsa_coded_cache *c);

// ---- device helpers ----------------------------------------------------------

constexpr float kLog2e = 1.4426950408889634f;

// 2^x; results below the smallest normal float are 0.
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// of AttendCodedArgs::sharing: the row may not add weights; the first, or a later,
// of several queries that add to one history's accumulators
constexpr uint32_t kBad = 1u, kFirstSharer = 2u, kLaterSharer = 4u;

// Query b's row.  ok: its count and T_b are in range (else it is empty).
struct Row {
    int groups, tail;   // complete groups; raw tokens behind them
    int T;              // visible tokens
    bool t_ok, ok;
};
__device__ __forceinline__ Row row_of(const AttendCodedArgs &a, int b)
{
    Row r;
    r.T = __ldg(a.visible + b);
    const int n = a.ids != nullptr ? __ldcg(a.n_ids + b) : r.T;
    r.t_ok = r.T >= 0 && r.T <= a.max_visible;
    r.ok = r.t_ok && n >= 0 && (a.ids == nullptr || n <= a.row_cap);
    r.groups = r.ok ? n / kGroup : 0;
    r.tail = r.ok ? n % kGroup : 0;
    return r;
}

}  // namespace qsa
