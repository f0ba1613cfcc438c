// api_rows.cu -- the extern "C" boundary of include/qsa_rows.h: argument
// validation before anything is enqueued, the launches.
#include <cuda_runtime.h>

#include "cache_internal.cuh"

namespace qsa {
namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool given(const void *p, size_t a) { return p != nullptr && aligned(p, a); }
qsa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? QSA_OK : QSA_ERR_CUDA; }

qsa_status check_ws(void *ws, size_t ws_bytes)
{
    static_assert(QSA_ROWS_WORKSPACE_BYTES == kWsAlign, "the error word's section");
    if (!given(ws, kWsAlign)) return QSA_ERR_INVALID_ARG;
    return ws_bytes < QSA_ROWS_WORKSPACE_BYTES ? QSA_ERR_WORKSPACE_TOO_SMALL : QSA_OK;
}

// Projection i of a family, if it is given: heads of `width`, written to `out`.
bool add(AppendFamily &f, int i, const qsa_projection &p, int heads, int width, int elem, const void *out)
{
    if (p.rows == nullptr) return true;
    if (!aligned(p.rows, 16) || !aligned(p.norm, 16) || !given(out, 16)) return false;
    if (int64_t(heads) * width > (1 << 30)) return false;  // (a row's elements are counted in 32 bits)
    if (p.stride < int64_t(heads) * width || p.stride > INT64_MAX / 65536 / 4 || p.stride * elem % 16 != 0) return false;
    f.rows[i] = p.rows;
    f.stride[i] = p.stride;
    f.norm[i] = p.norm;
    f.out[i] = static_cast<float *>(const_cast<void *>(out));
    f.heads[i] = heads;
    return true;
}

// Rows that are what is written: f32 queries that lie as they will.  Others would be overwritten before they are read.
bool in_place_only_as_it_lies(const AppendFamily &f, int elem, int width, int batch)
{
    for (int k = 0; k < 3; ++k) {
        if (f.heads[k] == 0 || f.rows[k] != f.out[k]) continue;
        if (k != 0 || elem != 4 || (batch > 1 && f.stride[k] != int64_t(f.heads[k]) * width)) return false;
    }
    return true;
}

bool turn(AppendFamily &f, const qsa_rotation &r, int width, const int32_t *positions)
{
    if (r.dims == 0) return true;
    if (r.dims < 0 || r.dims > width || r.dims % 8 != 0 || !given(r.freq, 4) || !given(positions, 4)) return false;
    if (r.pairing != QSA_PAIR_HALVES && r.pairing != QSA_PAIR_NEIGHBOURS) return false;
    f.dims = r.dims;
    f.freq = r.freq;
    f.neighbours = r.pairing == QSA_PAIR_NEIGHBOURS;
    return true;
}

}  // namespace
}  // namespace qsa

using namespace qsa;

extern "C" {

qsa_status qsa_append_tokens(const qsa_dims *dims, const qsa_inputs *in, const qsa_new_tokens *tokens, void *ws,
                             size_t ws_bytes, void *stream)
{
    if (!dims_valid(dims) || !in || !tokens) return QSA_ERR_INVALID_ARG;
    const qsa_new_tokens &t = *tokens;
    const bool kv = t.k.rows || t.v.rows, att = t.q.rows || kv, idx = t.q_idx.rows || t.idx_key.rows;
    if (!att && !idx) return QSA_ERR_INVALID_ARG;
    if (att && dims->head_dim != 64 && dims->head_dim != 128) return QSA_ERR_UNSUPPORTED_SHAPE;
    if (idx && dims->idx_dim != 32 && dims->idx_dim != 64) return QSA_ERR_UNSUPPORTED_SHAPE;
    if (t.type != QSA_ROWS_F32 && t.type != QSA_ROWS_BF16 && t.type != QSA_ROWS_F16) return QSA_ERR_INVALID_ARG;
    if (t.axes < 1 || t.axes > QSA_MAX_AXES || !(t.eps >= 0.0f) || t.v.norm != nullptr) return QSA_ERR_INVALID_ARG;
    if (!given(in->visible, 4)) return QSA_ERR_INVALID_ARG;
    if (kv && (!given(in->slot_map, 4) || !given(in->slot_offset, 8) || in->num_slots < 0)) return QSA_ERR_INVALID_ARG;
    if (t.idx_key.rows && !given(in->key_offset, 8)) return QSA_ERR_INVALID_ARG;
    AppendArgs a{};
    const int elem = t.type == QSA_ROWS_F32 ? 4 : 2, d = dims->head_dim, di = dims->idx_dim;
    if (!add(a.family[0], 0, t.q, dims->q_heads, d, elem, in->q) ||
        !add(a.family[0], 1, t.k, dims->kv_heads, d, elem, in->k_cache) ||
        !add(a.family[0], 2, t.v, dims->kv_heads, d, elem, in->v_cache) ||
        !add(a.family[1], 0, t.q_idx, dims->idx_heads, di, elem, in->q_idx) ||
        !add(a.family[1], 1, t.idx_key, 1, di, elem, in->idx_keys))
        return QSA_ERR_INVALID_ARG;
    if ((t.q.rows || t.k.rows) && !turn(a.family[0], t.turn, d, t.positions)) return QSA_ERR_INVALID_ARG;
    if (idx && !turn(a.family[1], t.turn_idx, di, t.positions)) return QSA_ERR_INVALID_ARG;
    const qsa_status st = check_ws(ws, ws_bytes);
    if (st != QSA_OK) return st;
    if (dims->batch == 0) return QSA_OK;
    for (int f = 0; f < 2; ++f)
        if (!in_place_only_as_it_lies(a.family[f], elem, f == 0 ? d : di, dims->batch)) return QSA_ERR_INVALID_ARG;
    a.positions = a.family[0].dims + a.family[1].dims > 0 ? t.positions : nullptr;  // (read only where something turns)
    a.visible = in->visible;
    a.slot_map = in->slot_map;
    a.slot_offset = in->slot_offset;
    a.key_offset = in->key_offset;
    a.num_slots = in->num_slots;
    a.eps = t.eps;
    a.axes = t.axes;
    a.batch = dims->batch;
    a.max_visible = dims->max_visible;
    a.err = static_cast<uint32_t *>(ws);
    const int sms = num_sms_of_current_device();
    if (sms <= 0) return QSA_ERR_CUDA;
    return from_cuda(launch_append(a, t.type, att ? d : 128, idx ? di : 64, sms, static_cast<cudaStream_t>(stream)));
}

qsa_status qsa_read_groups(const qsa_dims *dims, const qsa_inputs *in, const qsa_coded_cache *cache,
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
    if ((st = check_ws(ws, ws_bytes)) != QSA_OK) return st;
    CodeArgs a{in->k_cache, in->v_cache, in->num_slots, in->slot_map, in->slot_offset, group_begin, group_end,
               cache->codes, cache->scales, cache->num_blocks, cache->block_map, cache->block_offset, cache->format,
               dims->batch, dims->kv_heads, dims->head_dim, max_groups, g_max, static_cast<uint32_t *>(ws)};
    return from_cuda(launch_read_groups(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
