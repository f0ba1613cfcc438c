// evict.cu -- the groups that a history keeps, by accumulated attention
// (qsa_evict_select), and the history moved to its new place
// (qsa_evict_compact); include/qsa_cache.h.
#include <cooperative_groups.h>

#include "cache_internal.cuh"

namespace qsa {
namespace {

namespace cg = cooperative_groups;

// ---- membership ------------------------------------------------------------------
// The key of a weight orders as the weight does (order_key; a NaN below all), so
// the kept set of the n best by (weight descending, position ascending) is: every
// key above the n-th largest key K, and as many keys equal to K, lowest positions
// first, as are missing.  K comes from three counting passes (11, 11 and 10 bits),
// each over the keys that share the bits found so far.
//
// A cluster of CTAs takes one history, each CTA a contiguous slice of it; slices
// of up to kCached keys are read from memory once and kept in shared memory.  The
// CTAs count their slices and read one another's counts through distributed
// shared memory, so the whole choice is one launch with no workspace.  Latency
// bound: four bytes per group, a few cluster barriers.
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kPer = 4;                     // consecutive positions per thread in the emission
constexpr int kCached = 40960;              // keys a CTA keeps in shared memory at most
constexpr int kCluster = 8;

struct SelectSmem {
    uint32_t hist[kBins];
    uint32_t warp_sum[2][kWarps];
    uint32_t above, equal;                  // this slice's keys above and equal to K
    uint32_t bin, rest;
};

__device__ __forceinline__ uint32_t weight_key(float w)
{
    return w != w ? 0u : order_key(w);
}

// Sum over the block of (x, y), and the exclusive prefix of each thread.
__device__ __forceinline__ void block_scan2(SelectSmem &sm, uint32_t &x, uint32_t &y, uint32_t &tx, uint32_t &ty)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t x0 = x, y0 = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) {
            x += u;
            y += v;
        }
    }
    __syncthreads();
    if (lane == 31) {
        sm.warp_sum[0][warp] = x;
        sm.warp_sum[1][warp] = y;
    }
    __syncthreads();
    uint32_t px = 0, py = 0;
    tx = ty = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const uint32_t a = sm.warp_sum[0][w], b = sm.warp_sum[1][w];
        if (w < warp) {
            px += a;
            py += b;
        }
        tx += a;
        ty += b;
    }
    x += px - x0;
    y += py - y0;
}

__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictSelectArgs a, int cached)
{
    extern __shared__ __align__(16) uint32_t keys[];  // [cached]
    __shared__ SelectSmem sm;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = int(cluster.block_rank()), nr = int(cluster.num_blocks());
    const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    const int T = __ldg(a.visible + b);
    if (T < 0 || T > a.max_visible) {  // (the whole cluster leaves)
        if (rank == 0 && tid == 0) {
            a.n_kept[b] = 0;
            set_error(a.err, QSA_DEVERR_VISIBLE_RANGE);
        }
        return;
    }
    const int G = T / kGroup;
    int32_t *kept = a.kept + int64_t(b) * a.keep;
    if (rank == 0 && tid == 0) a.n_kept[b] = min(G, a.keep);
    if (G <= a.keep) {
        for (int g = rank * kThreads + tid; g < G; g += nr * kThreads) kept[g] = g;
        return;
    }
    int32_t *evicted = a.evicted != nullptr ? a.evicted + int64_t(b) * (a.max_visible / kGroup) : nullptr;
    // the choice is among the positions [lo, lo + n)
    const int lo = a.sink, n = G - a.sink - a.recent;
    const uint32_t need = uint32_t(a.keep - a.sink - a.recent);
    const float *w = a.weights + __ldg(a.weight_offset + b) + lo;
    const int slice = ((n + nr - 1) / nr + kPer - 1) / kPer * kPer;
    const int s0 = min(n, rank * slice), sn = min(n, s0 + slice) - s0;
    const bool in_smem = sn <= cached;
    if (in_smem) {
        for (int i = tid; i < sn; i += kThreads) keys[i] = weight_key(__ldg(w + s0 + i));
        __syncthreads();
    }
    auto key_at = [&](int i) { return in_smem ? keys[i] : weight_key(__ldg(w + s0 + i)); };

    // ---- K, the need-th largest key, and how many keys equal to it are kept ---------
    uint32_t K = 0xffffffffu, ties = 0;  // (no key is that large: nothing is kept)
    if (need > 0) {
        uint32_t rest = need, prefix = 0;
        int shift = 21, bits = 11;
        for (int pass = 0; pass < 3; ++pass) {
            for (int i = tid; i < kBins; i += kThreads) sm.hist[i] = 0;
            __syncthreads();
            const uint32_t above_mask = pass == 0 ? 0u : 0xffffffffu << (shift + bits);
            for (int i0 = 0; i0 < sn; i0 += kThreads) {
                const int i = i0 + tid;
                const uint32_t k = i < sn ? key_at(i) : 0u;
                const bool in = i < sn && (k & above_mask) == prefix;
                // many groups weigh the same (nothing, above all): a warp's equal bins are counted once
                const uint32_t bin = in ? (k >> shift) & ((1u << bits) - 1u) : 0xffffffffu;
                const uint32_t same = __match_any_sync(0xffffffffu, bin);
                if (in && lane == __ffs(same) - 1) atomicAdd(&sm.hist[bin], uint32_t(__popc(same)));
            }
            cluster.sync();
            // the counts of the whole history, from the top bin down: a thread takes four bins
            uint32_t c[kBins / kThreads], mine = 0, none = 0, total, unused;
#pragma unroll
            for (int j = 0; j < kBins / kThreads; ++j) {
                const int bin = kBins - 1 - (tid * (kBins / kThreads) + j);
                uint32_t sum = 0;
                for (int r = 0; r < nr; ++r) sum += cluster.map_shared_rank(sm.hist, r)[bin];
                c[j] = sum;
                mine += sum;
            }
            block_scan2(sm, mine, none, total, unused);  // mine: keys in the bins above this thread's
#pragma unroll
            for (int j = 0; j < kBins / kThreads; ++j) {
                if (mine < rest && rest <= mine + c[j]) {  // exactly one bin of one thread
                    sm.bin = uint32_t(kBins - 1 - (tid * (kBins / kThreads) + j));
                    sm.rest = rest - mine;
                }
                mine += c[j];
            }
            cluster.sync();  // every CTA has read the counts (and sm.bin is set)
            prefix |= sm.bin << shift;
            rest = sm.rest;
            bits = pass == 1 ? 10 : 11;
            shift -= bits;
        }
        K = prefix;
        ties = rest;
    }

    // ---- counts of the lower slices ----------------------------------------------------
    uint32_t gt = 0, eq = 0, tg, te;
    for (int i = tid; i < sn; i += kThreads) {
        const uint32_t k = key_at(i);
        gt += k > K;
        eq += k == K;
    }
    block_scan2(sm, gt, eq, tg, te);
    if (tid == 0) {
        sm.above = tg;
        sm.equal = te;
    }
    cluster.sync();
    uint32_t base_gt = 0, base_eq = 0;
    for (int r = 0; r < rank; ++r) {
        const SelectSmem *o = cluster.map_shared_rank(&sm, r);
        base_gt += o->above;
        base_eq += o->equal;
    }

    // ---- emission in ascending position ------------------------------------------------
    for (int i0 = 0; i0 < sn; i0 += kThreads * kPer) {
        const int first = i0 + tid * kPer;
        uint32_t k[kPer];
        gt = eq = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            k[j] = first + j < sn ? key_at(first + j) : 0u;
            if (first + j < sn) {
                gt += k[j] > K;
                eq += k[j] == K;
            }
        }
        block_scan2(sm, gt, eq, tg, te);
        uint32_t pg = base_gt + gt, pe = base_eq + eq;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (first + j >= sn) break;
            const int p = s0 + first + j;  // position - lo
            const uint32_t before = pg + min(pe, ties);
            const bool keep = k[j] > K || (k[j] == K && pe < ties);
            if (keep) kept[a.sink + before] = lo + p;
            else if (evicted != nullptr) evicted[uint32_t(p) - before] = lo + p;
            pg += k[j] > K;
            pe += k[j] == K;
        }
        base_gt += tg;
        base_eq += te;
    }
    if (rank == 0) {
        for (int g = tid; g < a.sink; g += kThreads) kept[g] = g;
        for (int j = tid; j < a.recent; j += kThreads) kept[a.keep - a.recent + j] = G - a.recent + j;
    }
    cluster.sync();  // no CTA leaves while another may read its shared memory
}

// ---- the move ------------------------------------------------------------------------
// Bound by memory: every kept row read once and written once (10*d_I*4 bytes of
// keys and 48 of maps and weights per group).  A warp takes a group: a lane's
// 16-byte pieces of the four raw rows and of the pooled row are all loaded
// before the first is stored.
constexpr int kMoveThreads = 256;
constexpr int kMoveWarps = kMoveThreads / 32;

template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_compact_kernel(const EvictCompactArgs a)
{
    constexpr int F4 = D / 4;               // 16-byte pieces of a row
    constexpr int kRaw = kGroup * F4 / 32;  // of the four raw rows, per lane
    const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    const int T = __ldg(a.src.visible + b), n = __ldg(a.n_kept + b);
    const int G = T / kGroup, tail = T % kGroup;
    if (T < 0 || T > a.max_visible || n < 0 || n > a.keep || n > G) {
        if (blockIdx.x == 0 && tid == 0) {
            a.dst.visible[b] = 0;
            set_error(a.err, T < 0 || T > a.max_visible ? QSA_DEVERR_VISIBLE_RANGE : QSA_DEVERR_ROW_RANGE);
        }
        return;
    }
    const qsa_history &s = a.src, &d = a.dst;
    if (blockIdx.x == 0) {
        if (tid == 0) d.visible[b] = kGroup * n + tail;
        if (tid < tail) {
            if (s.slot_map != nullptr)
                d.slot_map[__ldg(d.slot_offset + b) + kGroup * int64_t(n) + tid] =
                    __ldg(s.slot_map + __ldg(s.slot_offset + b) + kGroup * int64_t(G) + tid);
        }
        if (s.idx_keys != nullptr && tid < tail * F4)
            reinterpret_cast<float4 *>(d.idx_keys + (__ldg(d.key_offset + b) + kGroup * int64_t(n)) * D)[tid] =
                __ldg(reinterpret_cast<const float4 *>(s.idx_keys + (__ldg(s.key_offset + b) + kGroup * int64_t(G)) * D) + tid);
        if (s.weights != nullptr && tail > 0 && tid == 0)
            d.weights[__ldg(d.weight_offset + b) + n] = __ldg(s.weights + __ldg(s.weight_offset + b) + G);
    }
    const int32_t *kept = a.kept + int64_t(b) * a.keep;
    for (int i = int(blockIdx.x) * kMoveWarps + (tid >> 5); i < n; i += int(gridDim.x) * kMoveWarps) {
        const int g = __ldg(kept + i);
        const bool ok = g >= 0 && g < G;
        if (!ok && lane == 0) set_error(a.err, QSA_DEVERR_ROW_RANGE);
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        float4 raw[kRaw], pool = zero;
        int map = -1;
        float wt = 0.0f;
        if (s.idx_keys != nullptr) {
            const float4 *src = reinterpret_cast<const float4 *>(s.idx_keys + (__ldg(s.key_offset + b) + kGroup * int64_t(g)) * D);
#pragma unroll
            for (int j = 0; j < kRaw; ++j) raw[j] = ok ? __ldg(src + lane + 32 * j) : zero;
        }
        if (s.pooled != nullptr && lane < F4 && ok)  // piece p of the new row: its place depends on the position
            pool = __ldg(reinterpret_cast<const float4 *>(s.pooled + (__ldg(s.pool_offset + b) + g) * D) + (lane ^ (i & 7) ^ (g & 7)));
        if (ok) {
            if (s.slot_map != nullptr && lane < kGroup) map = __ldg(s.slot_map + __ldg(s.slot_offset + b) + kGroup * int64_t(g) + lane);
            if (s.block_map != nullptr && lane == kGroup) map = __ldg(s.block_map + __ldg(s.block_offset + b) + g);
            if (s.weights != nullptr && lane == kGroup + 1) wt = __ldg(s.weights + __ldg(s.weight_offset + b) + g);
        }
        if (s.idx_keys != nullptr) {
            float4 *dst = reinterpret_cast<float4 *>(d.idx_keys + (__ldg(d.key_offset + b) + kGroup * int64_t(i)) * D);
#pragma unroll
            for (int j = 0; j < kRaw; ++j) dst[lane + 32 * j] = raw[j];
        }
        if (s.pooled != nullptr && lane < F4)
            reinterpret_cast<float4 *>(d.pooled + (__ldg(d.pool_offset + b) + i) * D)[lane] = pool;
        if (s.slot_map != nullptr && lane < kGroup) d.slot_map[__ldg(d.slot_offset + b) + kGroup * int64_t(i) + lane] = map;
        if (s.block_map != nullptr && lane == kGroup) d.block_map[__ldg(d.block_offset + b) + i] = map;
        if (s.weights != nullptr && lane == kGroup + 1) d.weights[__ldg(d.weight_offset + b) + i] = wt;
    }
}

}  // namespace

cudaError_t launch_evict_select(const EvictSelectArgs &a, cudaStream_t s)
{
    if (a.batch == 0) return cudaSuccess;
    static bool attr_done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_done[dev]) {
        e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCached * 4);
        if (e != cudaSuccess) return e;
        attr_done[dev] = true;
    }
    const int groups = a.max_visible / kGroup;
    const int nr = groups <= 4096 ? 1 : kCluster;
    const int slice = ((groups + nr - 1) / nr + kPer - 1) / kPer * kPer;
    const int cached = slice < kCached ? slice : kCached;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(nr), unsigned(a.batch));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = size_t(cached) * 4;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(nr);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_select_kernel, a, cached);
}

cudaError_t launch_evict_compact(const EvictCompactArgs &a, int num_sms, cudaStream_t s)
{
    if (a.batch == 0) return cudaSuccess;
    const int most = a.keep < a.max_visible / kGroup ? a.keep : a.max_visible / kGroup;
    const int blocks = (most + kMoveWarps - 1) / kMoveWarps;
    const int cap = 64 * num_sms;
    const dim3 grid(unsigned(blocks < 1 ? 1 : blocks < cap ? blocks : cap), unsigned(a.batch));
    if (a.idx_dim == 64) evict_compact_kernel<64><<<grid, kMoveThreads, 0, s>>>(a);
    else if (a.idx_dim == 32) evict_compact_kernel<32><<<grid, kMoveThreads, 0, s>>>(a);
    else return cudaErrorInvalidValue;
    return cudaGetLastError();
}

}  // namespace qsa
