// api_cache.cu -- the extern "C" boundary of include/qsa_cache.h: argument
// validation before anything is enqueued, the workspace layout, the launches.
#include <cuda_runtime.h>

#include "cache_internal.cuh"

namespace qsa {

CodedLayout make_coded_layout(const qsa_dims *d, bool whole, bool weights)
{
    CodedLayout C{};
    C.base = make_layout(d);
    const int g_max = d->max_visible / kGroup;
    const size_t heads = size_t(d->batch) * size_t(d->q_heads);
    size_t off = C.base.total;
    if (whole) {
        C.nparts = coded_max_runs(g_max, true, d->q_heads / d->kv_heads) + 1;
        C.off_part_m = off;
        off = align_up(off + heads * size_t(C.nparts) * 4, kWsAlign);
        C.off_part_l = off;
        off = align_up(off + heads * size_t(C.nparts) * 4, kWsAlign);
        C.off_part_acc = off;
        off = align_up(off + heads * size_t(C.nparts) * size_t(d->head_dim) * 4, kWsAlign);
    } else {  // selected rows: the partial states of qsa_attend's layout
        static_assert(QSA_MAX_BUDGET / kCodedRunRows + 1 <= kAttendParts, "runs of the longest row, and its tail");
        C.nparts = C.base.nparts;
        C.off_part_m = C.base.off_part_m;
        C.off_part_l = C.base.off_part_l;
        C.off_part_acc = C.base.off_part_acc;
    }
    if (weights) {
        int groups = d->budget_groups;
        if (whole && g_max > groups) groups = g_max;  // (serves selected rows too)
        C.mass_stride = (groups + 3) / 4 * 4;
        C.off_mass = off;
        off = align_up(off + heads * size_t(C.mass_stride) * 4, kWsAlign);
        C.off_mref = off;
        off = align_up(off + heads * size_t(C.mass_stride / 4) * 4, kWsAlign);
        C.off_stat = off;
        off = align_up(off + heads * 8, kWsAlign);
        C.off_sharing = off;
        off = align_up(off + size_t(d->batch) * 4, kWsAlign);
        C.off_tail = off;
        off = align_up(off + size_t(d->batch) * 4, kWsAlign);
        C.map_stride = int(C.base.score_stride);
    }
    C.total = off;
    return C;
}

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool given(const void *p, size_t a) { return p != nullptr && aligned(p, a); }
qsa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? QSA_OK : QSA_ERR_CUDA; }

template <typename T>
T *at(void *ws, size_t off)
{
    return reinterpret_cast<T *>(static_cast<unsigned char *>(ws) + off);
}

qsa_status check_ws(void *ws, size_t ws_bytes, size_t need)
{
    if (!given(ws, kWsAlign)) return QSA_ERR_INVALID_ARG;
    return ws_bytes < need ? QSA_ERR_WORKSPACE_TOO_SMALL : QSA_OK;
}

// The f32 cache behind the slot map.
qsa_status check_rows(const qsa_inputs *in)
{
    if (!in || !given(in->k_cache, 16) || !given(in->v_cache, 16) || !given(in->slot_map, 4) ||
        !given(in->slot_offset, 8) || in->num_slots < 0)
        return QSA_ERR_INVALID_ARG;
    return QSA_OK;
}

qsa_status check_cache(const qsa_coded_cache *c)
{
    if (!c || !given(c->codes, 16) || !given(c->scales, 16) || !given(c->block_map, 4) || !given(c->block_offset, 8) ||
        c->num_blocks < 0)
        return QSA_ERR_INVALID_ARG;
    if (c->format != QSA_CODE_E4M3 && c->format != QSA_CODE_INT8) return QSA_ERR_INVALID_ARG;
    return QSA_OK;
}

qsa_status check_attend(const qsa_dims *d, const qsa_inputs *in, const qsa_coded_cache *cache, const float *out,
                        const float *weights, const int64_t *weight_offset)
{
    if (!attend_coded_shape_supported(d->head_dim, d->q_heads, d->kv_heads)) return QSA_ERR_UNSUPPORTED_SHAPE;
    qsa_status st;
    if ((st = check_rows(in)) != QSA_OK) return st;
    if (!given(in->q, 16) || !given(in->visible, 4) || !given(out, 16)) return QSA_ERR_INVALID_ARG;
    if ((weights == nullptr) != (weight_offset == nullptr)) return QSA_ERR_INVALID_ARG;
    if (weights && (!aligned(weights, 4) || !aligned(weight_offset, 8))) return QSA_ERR_INVALID_ARG;
    return check_cache(cache);
}

AttendCodedArgs attend_args(const qsa_dims *d, const qsa_inputs *in, const qsa_coded_cache *cache, const int32_t *ids,
                            const int32_t *n_ids, float *out, float *weights, const int64_t *weight_offset, void *ws,
                            const CodedLayout &C)
{
    AttendCodedArgs a{};
    a.q = in->q;
    a.visible = in->visible;
    a.ids = ids;
    a.n_ids = n_ids;
    a.codes = cache->codes;
    a.scales = cache->scales;
    a.num_blocks = cache->num_blocks;
    a.block_map = cache->block_map;
    a.block_offset = cache->block_offset;
    a.k_cache = in->k_cache;
    a.v_cache = in->v_cache;
    a.num_slots = in->num_slots;
    a.slot_map = in->slot_map;
    a.slot_offset = in->slot_offset;
    a.out = out;
    a.part_m = at<float>(ws, C.off_part_m);
    a.part_l = at<float>(ws, C.off_part_l);
    a.part_acc = at<float>(ws, C.off_part_acc);
    if (weights) {
        a.mass = at<float>(ws, C.off_mass);
        a.mref = at<float>(ws, C.off_mref);
        a.stat = at<float>(ws, C.off_stat);
        a.sharing = at<uint32_t>(ws, C.off_sharing);
        if (d->batch > 1) a.share_map = at<float>(ws, C.base.off_scores);  // (one query shares with nobody)
        a.tail_share = at<float>(ws, C.off_tail);
        a.map_stride = C.map_stride;
        a.weights = weights;
        a.weight_offset = weight_offset;
    }
    a.format = cache->format;
    a.batch = d->batch;
    a.q_heads = d->q_heads;
    a.kv_heads = d->kv_heads;
    a.head_dim = d->head_dim;
    a.row_cap = C.base.row_cap;
    a.nparts = C.nparts;
    a.mass_stride = C.mass_stride;
    a.max_visible = d->max_visible;
    a.scale = d->scale;
    a.err = at<uint32_t>(ws, C.base.off_err);
    return a;
}

}  // namespace
}  // namespace qsa

using namespace qsa;

extern "C" {

size_t qsa_coded_workspace_size(const qsa_dims *dims, int32_t whole_history, int32_t with_weights)
{
    if (!dims_valid(dims)) return 0;
    return make_coded_layout(dims, whole_history != 0, with_weights != 0).total;
}

qsa_status qsa_code_groups(const qsa_dims *dims, const qsa_inputs *in, const qsa_coded_cache *cache,
                           const int32_t *group_begin, const int32_t *group_end, int32_t max_groups, void *ws,
                           size_t ws_bytes, void *stream)
{
    if (!dims_valid(dims)) return QSA_ERR_INVALID_ARG;
    if (dims->head_dim != 64 && dims->head_dim != 128) return QSA_ERR_UNSUPPORTED_SHAPE;
    qsa_status st;
    if ((st = check_rows(in)) != QSA_OK || (st = check_cache(cache)) != QSA_OK) return st;
    if (!given(group_begin, 4) || !given(group_end, 4)) return QSA_ERR_INVALID_ARG;
    const int32_t g_max = dims->max_visible / kGroup;
    if (max_groups < 0 || max_groups > g_max) return QSA_ERR_INVALID_ARG;
    const Layout L = make_layout(dims);
    if ((st = check_ws(ws, ws_bytes, L.total)) != QSA_OK) return st;
    CodeArgs a{in->k_cache, in->v_cache, in->num_slots, in->slot_map, in->slot_offset, group_begin, group_end,
               cache->codes, cache->scales, cache->num_blocks, cache->block_map, cache->block_offset, cache->format,
               dims->batch, dims->kv_heads, dims->head_dim, max_groups, g_max, at<uint32_t>(ws, L.off_err)};
    return from_cuda(launch_code_groups(a, static_cast<cudaStream_t>(stream)));
}

qsa_status qsa_attend_coded(const qsa_dims *dims, const qsa_inputs *in, const qsa_coded_cache *cache,
                            const int32_t *ids, const int32_t *n_ids, float *out, float *weights,
                            const int64_t *weight_offset, void *ws, size_t ws_bytes, void *stream)
{
    if (!dims_valid(dims)) return QSA_ERR_INVALID_ARG;
    qsa_status st;
    if ((st = check_attend(dims, in, cache, out, weights, weight_offset)) != QSA_OK) return st;
    if ((ids == nullptr) != (n_ids == nullptr) || !aligned(ids, 4) || !aligned(n_ids, 4)) return QSA_ERR_INVALID_ARG;
    const CodedLayout C = make_coded_layout(dims, ids == nullptr, weights != nullptr);
    if ((st = check_ws(ws, ws_bytes, C.total)) != QSA_OK) return st;
    const AttendCodedArgs a = attend_args(dims, in, cache, ids, n_ids, out, weights, weight_offset, ws, C);
    return from_cuda(launch_attend_coded(a, static_cast<cudaStream_t>(stream)));
}

qsa_status qsa_decode_coded(const qsa_dims *dims, const qsa_inputs *in, const qsa_coded_cache *cache,
                            const float *pooled, const int64_t *pool_offset, int32_t *ids, int32_t *n_ids, float *out,
                            float *weights, const int64_t *weight_offset, void *ws, size_t ws_bytes, void *stream)
{
    if (!dims_valid(dims)) return QSA_ERR_INVALID_ARG;
    if (!score_shape_supported(dims->idx_heads, dims->idx_dim)) return QSA_ERR_UNSUPPORTED_SHAPE;
    qsa_status st;
    if ((st = check_attend(dims, in, cache, out, weights, weight_offset)) != QSA_OK) return st;
    if (!given(in->q_idx, 16) || (pooled == nullptr) != (pool_offset == nullptr)) return QSA_ERR_INVALID_ARG;
    if (pooled ? !aligned(pooled, 16) || !aligned(pool_offset, 8) : !given(in->idx_keys, 16) || !given(in->key_offset, 8))
        return QSA_ERR_INVALID_ARG;
    if (!given(ids, 4) || !given(n_ids, 4)) return QSA_ERR_INVALID_ARG;
    const CodedLayout C = make_coded_layout(dims, false, weights != nullptr);
    if ((st = check_ws(ws, ws_bytes, C.total)) != QSA_OK) return st;
    if (dims->batch == 0) return QSA_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((st = score_and_select(dims, in, pooled, pool_offset, ws, C.base, s)) != QSA_OK) return st;
    // the attention reads the rows in the workspace and stores the caller's copy with its output
    AttendCodedArgs a = attend_args(dims, in, cache, at<int32_t>(ws, C.base.off_ids), at<int32_t>(ws, C.base.off_nids),
                                    out, weights, weight_offset, ws, C);
    a.ids_out = ids;
    a.n_ids_out = n_ids;
    return from_cuda(launch_attend_coded(a, s));
}

qsa_status qsa_evict_select(const qsa_dims *dims, const int32_t *visible, const float *weights,
                            const int64_t *weight_offset, int32_t keep_groups, int32_t sink_groups,
                            int32_t recent_groups, int32_t *kept, int32_t *n_kept, int32_t *evicted, void *ws,
                            size_t ws_bytes, void *stream)
{
    if (!dims_valid(dims)) return QSA_ERR_INVALID_ARG;
    if (!given(visible, 4) || !given(weights, 4) || !given(weight_offset, 8) || !given(kept, 4) || !given(n_kept, 4) ||
        !aligned(evicted, 4))
        return QSA_ERR_INVALID_ARG;
    if (keep_groups < 1 || keep_groups > QSA_MAX_VISIBLE / kGroup || sink_groups < 0 || recent_groups < 0 ||
        sink_groups > keep_groups || recent_groups > keep_groups - sink_groups)
        return QSA_ERR_INVALID_ARG;
    const Layout L = make_layout(dims);
    qsa_status st;
    if ((st = check_ws(ws, ws_bytes, L.total)) != QSA_OK) return st;
    EvictSelectArgs a{visible, weights, weight_offset, kept, n_kept, evicted, dims->batch, dims->max_visible,
                      keep_groups, sink_groups, recent_groups, at<uint32_t>(ws, L.off_err)};
    return from_cuda(launch_evict_select(a, static_cast<cudaStream_t>(stream)));
}

qsa_status qsa_evict_compact(const qsa_dims *dims, int32_t keep_groups, const int32_t *kept, const int32_t *n_kept,
                             const qsa_history *src, const qsa_history *dst, void *ws, size_t ws_bytes, void *stream)
{
    if (!dims_valid(dims)) return QSA_ERR_INVALID_ARG;
    if (dims->idx_dim != 32 && dims->idx_dim != 64) return QSA_ERR_UNSUPPORTED_SHAPE;
    if (!given(kept, 4) || !given(n_kept, 4) || !src || !dst) return QSA_ERR_INVALID_ARG;
    if (keep_groups < 1 || keep_groups > QSA_MAX_VISIBLE / kGroup) return QSA_ERR_INVALID_ARG;
    if (!given(src->visible, 4) || !given(dst->visible, 4) || src->visible == dst->visible) return QSA_ERR_INVALID_ARG;
    // a member that one history has, the other has too, with both offsets and elsewhere
    auto pair_ok = [](const void *s, const void *so, const void *d, const void *dof, size_t align) {
        if (s == nullptr && d == nullptr) return true;
        return given(s, align) && given(d, align) && s != d && given(so, 8) && given(dof, 8);
    };
    if (!pair_ok(src->idx_keys, src->key_offset, dst->idx_keys, dst->key_offset, 16) ||
        !pair_ok(src->pooled, src->pool_offset, dst->pooled, dst->pool_offset, 16) ||
        !pair_ok(src->slot_map, src->slot_offset, dst->slot_map, dst->slot_offset, 4) ||
        !pair_ok(src->block_map, src->block_offset, dst->block_map, dst->block_offset, 4) ||
        !pair_ok(src->weights, src->weight_offset, dst->weights, dst->weight_offset, 4))
        return QSA_ERR_INVALID_ARG;
    const Layout L = make_layout(dims);
    qsa_status st;
    if ((st = check_ws(ws, ws_bytes, L.total)) != QSA_OK) return st;
    if (dims->batch == 0) return QSA_OK;
    const int sms = num_sms_of_current_device();
    if (sms <= 0) return QSA_ERR_CUDA;
    EvictCompactArgs a{kept, n_kept, *src, *dst, dims->batch, dims->max_visible, keep_groups, dims->idx_dim,
                       at<uint32_t>(ws, L.off_err)};
    return from_cuda(launch_evict_compact(a, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
