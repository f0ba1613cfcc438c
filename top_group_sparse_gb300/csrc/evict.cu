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
// shared memory -- those also say how many keys above and equal to K the slices
// before it hold, where a CTA's output begins -- so the whole choice is one launch
// with one cluster barrier per pass and no workspace.  Latency bound: 65,536
// groups 25.6 us, of which a cluster that has next to nothing to do takes 13; so
// histories of up to kOneCta groups take one CTA and no cluster (6.0 us).
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kPer = 8;                     // consecutive positions per thread in the emission
constexpr int kCached = 40960;              // keys a CTA keeps in shared memory at most
constexpr int kCluster = 8;
constexpr int kOneCta = 4096;               // histories of up to so many groups: one CTA, no cluster

struct SelectSmem {
    alignas(16) uint32_t hist[3][kBins];    // one per pass: a pass needs no barrier behind the others' reads
    uint32_t warp_sum[2][kWarps];           // by turns: a scan needs one barrier
    uint32_t bin, rest, equal;
};

__device__ __forceinline__ uint32_t weight_key(float w)
{
    return w != w ? 0u : order_key(w);
}

// The exclusive prefix of x over the block, and the sum; one barrier.
__device__ __forceinline__ uint32_t block_scan(SelectSmem &sm, int &turn, uint32_t x, uint32_t &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) sm.warp_sum[turn][warp] = incl;
    __syncthreads();
    uint32_t sums = lane < kWarps ? sm.warp_sum[turn][lane] : 0u;
    turn ^= 1;
#pragma unroll
    for (int o = 1; o < kWarps; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, sums, o);
        if (lane >= o) sums += u;
    }
    total = __shfl_sync(0xffffffffu, sums, kWarps - 1);
    const uint32_t before = __shfl_sync(0xffffffffu, sums, warp > 0 ? warp - 1 : 0);
    return (warp > 0 ? before : 0u) + incl - x;
}

template <int kRanks>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictSelectArgs a, int cached)
{
    extern __shared__ __align__(16) uint32_t keys[];  // [cached]
    __shared__ SelectSmem sm;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = kRanks == 1 ? 0 : int(cluster.block_rank());
    const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    wait_for_predecessor();
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
        for (int g = rank * kThreads + tid; g < G; g += kRanks * kThreads) kept[g] = g;
        return;
    }
    int32_t *evicted = a.evicted != nullptr ? a.evicted + int64_t(b) * (a.max_visible / kGroup) : nullptr;
    // the choice is among the positions [lo, lo + n)
    const int lo = a.sink, n = G - a.sink - a.recent;
    const uint32_t need = uint32_t(a.keep - a.sink - a.recent);
    const float *w = a.weights + __ldg(a.weight_offset + b) + lo;
    const int slice = ((n + kRanks - 1) / kRanks + kPer - 1) / kPer * kPer;
    const int s0 = min(n, rank * slice), sn = min(n, s0 + slice) - s0;
    const bool in_smem = sn <= cached;
    if (in_smem) {
#pragma unroll 8
        for (int i = tid; i < sn; i += kThreads) keys[i] = weight_key(__ldg(w + s0 + i));
    }
    auto key_at = [&](int i) { return in_smem ? keys[i] : weight_key(__ldg(w + s0 + i)); };
#pragma unroll
    for (int i = 0; i < kBins / kThreads; ++i)
        for (auto &counts : sm.hist) counts[tid + i * kThreads] = 0;
    __syncthreads();

    // ---- K, the need-th largest key, and how many keys equal to it are kept; the keys
    // above and equal to K in the slices before this one ----------------------------------
    uint32_t K = 0xffffffffu, ties = 0;  // (no key is that large: nothing is kept)
    uint32_t base_gt = 0, base_eq = 0;
    int turn = 0;
    if (need > 0) {
        uint32_t rest = need, prefix = 0, my_gt = 0;
        int shift = 21, bits = 11;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            uint32_t *my_hist = sm.hist[pass];
            const uint32_t above_mask = pass == 0 ? 0u : 0xffffffffu << (shift + bits);
#pragma unroll 4
            for (int i0 = 0; i0 < sn; i0 += kThreads) {
                const int i = i0 + tid;
                const uint32_t k = i < sn ? key_at(i) : 0u;
                const bool in = i < sn && (k & above_mask) == prefix;
                if (!__any_sync(0xffffffffu, in)) continue;
                // many groups weigh the same (nothing, above all): a warp's equal bins are counted once
                const uint32_t bin = in ? (k >> shift) & ((1u << bits) - 1u) : 0xffffffffu;
                const uint32_t same = __match_any_sync(0xffffffffu, bin);
                if (in && lane == __ffs(same) - 1) atomicAdd(&my_hist[bin], uint32_t(__popc(same)));
            }
            if constexpr (kRanks == 1) __syncthreads();
            else cluster.sync();
            // the counts of the whole history, from the top bin down: a thread takes four bins
            constexpr int kMine = kBins / kThreads;
            static_assert(kMine == 4, "a thread's bins are one 16-byte piece");
            const int first_bin = kBins - kMine * (tid + 1);
            uint4 v[kRanks];
#pragma unroll
            for (int r = 0; r < kRanks; ++r)
                v[r] = *reinterpret_cast<const uint4 *>((kRanks == 1 ? my_hist : cluster.map_shared_rank(my_hist, r)) + first_bin);
            uint32_t c[kMine] = {0, 0, 0, 0}, before[kMine] = {0, 0, 0, 0};  // of all slices, of the slices before this one
#pragma unroll
            for (int r = 0; r < kRanks; ++r) {
                const uint32_t x[kMine] = {v[r].w, v[r].z, v[r].y, v[r].x};
#pragma unroll
                for (int j = 0; j < kMine; ++j) {
                    c[j] += x[j];
                    if (r < rank) before[j] += x[j];
                }
            }
            uint32_t total;
            uint32_t above = block_scan(sm, turn, (c[0] + c[1]) + (c[2] + c[3]), total);  // keys in the bins above this thread's
#pragma unroll
            for (int j = 0; j < kMine; ++j) {
                if (above + c[j] < rest) my_gt += before[j];  // a bin above K's
                if (above < rest && rest <= above + c[j]) {   // K's bin: exactly one bin of one thread
                    sm.bin = uint32_t(first_bin + kMine - 1 - j);
                    sm.rest = rest - above;
                    sm.equal = before[j];
                }
                above += c[j];
            }
            __syncthreads();
            prefix |= sm.bin << shift;
            rest = sm.rest;
            bits = pass == 1 ? 10 : 11;
            shift -= bits;
        }
        K = prefix;
        ties = rest;
        base_eq = sm.equal;
        if constexpr (kRanks > 1) (void)block_scan(sm, turn, my_gt, base_gt);
    }
    // no CTA leaves while another may read its counts: this one has read the others'
    if constexpr (kRanks > 1) cluster.barrier_arrive();

    // ---- emission in ascending position ------------------------------------------------
    for (int i0 = 0; i0 < sn; i0 += kThreads * kPer) {
        const int first = i0 + tid * kPer;
        uint32_t k[kPer], gt = 0, eq = 0, total;
        if (in_smem) {  // (16-byte reads; what is behind the slice is not used)
#pragma unroll
            for (int j = 0; j < kPer; j += 4) {
                const uint4 x = first + j < sn ? *reinterpret_cast<const uint4 *>(keys + first + j) : make_uint4(0, 0, 0, 0);
                k[j] = x.x, k[j + 1] = x.y, k[j + 2] = x.z, k[j + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j) k[j] = first + j < sn ? weight_key(__ldg(w + s0 + first + j)) : 0u;
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (first + j < sn) {
                gt += k[j] > K;
                eq += k[j] == K;
            }
        }
        static_assert(kThreads * kPer < 65536, "both counts of a turn in one word");
        const uint32_t before = block_scan(sm, turn, gt | (eq << 16), total);
        uint32_t pg = base_gt + (before & 0xffffu), pe = base_eq + (before >> 16);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (first + j >= sn) break;
            const int p = s0 + first + j;  // position - lo
            const uint32_t at = pg + min(pe, ties);  // kept before it
            const bool keep = k[j] > K || (k[j] == K && pe < ties);
            if (keep) kept[a.sink + at] = lo + p;
            else if (evicted != nullptr) evicted[uint32_t(p) - at] = lo + p;
            pg += k[j] > K;
            pe += k[j] == K;
        }
        base_gt += total & 0xffffu;
        base_eq += total >> 16;
    }
    if (rank == 0) {
        for (int g = tid; g < a.sink; g += kThreads) kept[g] = g;
        for (int j = tid; j < a.recent; j += kThreads) kept[a.keep - a.recent + j] = G - a.recent + j;
    }
    if constexpr (kRanks > 1) cluster.barrier_wait();
}

// ---- the move ------------------------------------------------------------------------
// Bound by memory: every kept row read once and written once (10*d_I*4 bytes of
// keys and 48 of maps and weights per group).  A warp takes kTake groups at a
// time: a lane's 16-byte pieces of all their rows are loaded before the first is
// stored, and the next groups' positions while they are on their way.  Eight
// histories of 65,536 groups cut to half: 24 CTAs per SM 104 us (6.6 TB/s), 16 107
// us, 12 109 us; one CTA per 8 groups, each with its three dependent loads before
// the first row, 117 us.
constexpr int kMoveThreads = 256;
constexpr int kMoveWarps = kMoveThreads / 32;
constexpr int kTake = 2;
constexpr int kMoveCtas = 24;               // per SM, over the whole batch

template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_compact_kernel(const EvictCompactArgs a)
{
    constexpr int F4 = D / 4;               // 16-byte pieces of a row
    constexpr int kRaw = kGroup * F4 / 32;  // of the four raw rows, per lane
    const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    wait_for_predecessor();
    const int T = __ldg(a.src.visible + b), n = __ldg(a.n_kept + b);
    const int G = T / kGroup, tail = T % kGroup;
    if (T < 0 || T > a.max_visible || n < 0 || n > a.keep || n > G) {
        if (blockIdx.x == 0 && tid == 0) {
            a.dst.visible[b] = 0;
            set_error(a.err, T < 0 || T > a.max_visible ? QSA_DEVERR_VISIBLE_RANGE : QSA_DEVERR_ROW_RANGE);
        }
        return;
    }
    // query b's regions (16-byte pieces for the keys); a member that is not moved stays NULL
    const qsa_history &s = a.src, &d = a.dst;
    auto region = [&](auto *p, const int64_t *offset, int64_t row) { return p == nullptr ? p : p + __ldg(offset + b) * row; };
    const float4 *s_raw = reinterpret_cast<const float4 *>(region(s.idx_keys, s.key_offset, D));
    float4 *d_raw = reinterpret_cast<float4 *>(region(d.idx_keys, d.key_offset, D));
    const float4 *s_pool = reinterpret_cast<const float4 *>(region(s.pooled, s.pool_offset, D));
    float4 *d_pool = reinterpret_cast<float4 *>(region(d.pooled, d.pool_offset, D));
    // a lane's entry of the maps and weights, as 32-bit words: lanes 0-3 the slots of a
    // group, lane 4 its block, lane 5 its weight
    const uint32_t *s_map = nullptr;
    uint32_t *d_map = nullptr;
    int per = 0;  // words per group
    if (lane < kGroup && s.slot_map != nullptr) {
        s_map = reinterpret_cast<const uint32_t *>(region(s.slot_map, s.slot_offset, 1)) + lane;
        d_map = reinterpret_cast<uint32_t *>(region(d.slot_map, d.slot_offset, 1)) + lane;
        per = kGroup;
    } else if (lane == kGroup && s.block_map != nullptr) {
        s_map = reinterpret_cast<const uint32_t *>(region(s.block_map, s.block_offset, 1));
        d_map = reinterpret_cast<uint32_t *>(region(d.block_map, d.block_offset, 1));
        per = 1;
    } else if (lane == kGroup + 1 && s.weights != nullptr) {
        s_map = reinterpret_cast<const uint32_t *>(region(s.weights, s.weight_offset, 1));
        d_map = reinterpret_cast<uint32_t *>(region(d.weights, d.weight_offset, 1));
        per = 1;
    }
    if (blockIdx.x == 0 && tid < 32) {  // the raw tail, by the first warp
        if (lane == 0) d.visible[b] = kGroup * n + tail;
        if (lane < tail && s_map != nullptr) d_map[int64_t(kGroup) * n] = __ldg(s_map + int64_t(kGroup) * G);
        if (lane == kGroup + 1 && tail > 0 && s_map != nullptr) d_map[n] = __ldg(s_map + G);
        if (s_raw != nullptr)
            for (int e = lane; e < tail * F4; e += 32) d_raw[int64_t(kGroup * F4) * n + e] = __ldg(s_raw + int64_t(kGroup * F4) * G + e);
    }
    const int32_t *kept = a.kept + int64_t(b) * a.keep;
    const uint32_t none = lane == kGroup + 1 ? 0u : 0xffffffffu;  // of a bad position: weight 0, map entries -1
    const int stride = int(gridDim.x) * kMoveWarps * kTake;
    int i0 = (int(blockIdx.x) * kMoveWarps + (tid >> 5)) * kTake;
    int next[kTake];
#pragma unroll
    for (int u = 0; u < kTake; ++u) next[u] = i0 + u < n ? __ldg(kept + i0 + u) : 0;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    for (; i0 < n; i0 += stride) {
        float4 raw[kTake][kRaw], pool[kTake];
        uint32_t map[kTake];
        int g[kTake];
        bool ok[kTake];
#pragma unroll
        for (int u = 0; u < kTake; ++u) {
            g[u] = next[u];
            ok[u] = i0 + u < n && g[u] >= 0 && g[u] < G;
            if (i0 + u < n && !ok[u] && lane == 0) set_error(a.err, QSA_DEVERR_ROW_RANGE);
            if (s_raw != nullptr) {
#pragma unroll
                for (int j = 0; j < kRaw; ++j) raw[u][j] = ok[u] ? __ldg(s_raw + int64_t(kGroup * F4) * g[u] + lane + 32 * j) : zero;
            }
            // piece p of the new row: its place depends on the position.  (Through L2: the append
            // of pooled keys lets its successor start before it has written.)
            if (s_pool != nullptr && lane < F4)
                pool[u] = ok[u] ? __ldcg(s_pool + int64_t(F4) * g[u] + (lane ^ ((i0 + u) & 7) ^ (g[u] & 7))) : zero;
            if (s_map != nullptr) map[u] = ok[u] ? __ldg(s_map + int64_t(per) * g[u]) : none;
        }
#pragma unroll
        for (int u = 0; u < kTake; ++u) next[u] = i0 + stride + u < n ? __ldg(kept + i0 + stride + u) : 0;
#pragma unroll
        for (int u = 0; u < kTake; ++u) {
            const int64_t i = i0 + u;
            if (i >= n) break;
            if (s_raw != nullptr) {
#pragma unroll
                for (int j = 0; j < kRaw; ++j) d_raw[int64_t(kGroup * F4) * i + lane + 32 * j] = raw[u][j];
            }
            if (s_pool != nullptr && lane < F4) d_pool[int64_t(F4) * i + lane] = pool[u];
            if (s_map != nullptr) d_map[int64_t(per) * i] = map[u];
        }
    }
}

}  // namespace

template <int kRanks>
static cudaError_t launch_select_t(const EvictSelectArgs &a, cudaStream_t s)
{
    static bool attr_done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_done[dev]) {
        e = cudaFuncSetAttribute(evict_select_kernel<kRanks>, cudaFuncAttributeMaxDynamicSharedMemorySize, kCached * 4);
        if (e != cudaSuccess) return e;
        attr_done[dev] = true;
    }
    const int groups = a.max_visible / kGroup;
    const int slice = ((groups + kRanks - 1) / kRanks + kPer - 1) / kPer * kPer;
    const int cached = slice < kCached ? slice : kCached;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kRanks, unsigned(a.batch));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = size_t(cached) * 4;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kRanks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kRanks > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, evict_select_kernel<kRanks>, a, cached);
}

cudaError_t launch_evict_select(const EvictSelectArgs &a, cudaStream_t s)
{
    if (a.batch == 0) return cudaSuccess;
    return a.max_visible / kGroup <= kOneCta ? launch_select_t<1>(a, s) : launch_select_t<kCluster>(a, s);
}

cudaError_t launch_evict_compact(const EvictCompactArgs &a, int num_sms, cudaStream_t s)
{
    if (a.batch == 0) return cudaSuccess;
    const int most = a.keep < a.max_visible / kGroup ? a.keep : a.max_visible / kGroup;
    const int per_cta = kMoveWarps * kTake;
    const int blocks = (most + per_cta - 1) / per_cta, cap = kMoveCtas * num_sms / a.batch + 1;
    const dim3 grid(unsigned(blocks < 1 ? 1 : blocks < cap ? blocks : cap), unsigned(a.batch));
    if (a.idx_dim == 64) return launch_kernel(evict_compact_kernel<64>, grid, dim3(kMoveThreads), 0, s, true, a);
    if (a.idx_dim == 32) return launch_kernel(evict_compact_kernel<32>, grid, dim3(kMoveThreads), 0, s, true, a);
    return cudaErrorInvalidValue;
}

}  // namespace qsa
