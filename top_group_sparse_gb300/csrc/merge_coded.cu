// merge_coded.cu -- the second half of qsa_attend_coded (include/qsa_cache.h):
// the states of a row's runs merged, and the attention that each group received
// added to its accumulator.
#include <type_traits>

#include "cache_internal.cuh"

namespace qsa {
namespace {

// ---- the runs of a row merged in run order -----------------------------------------------
// Per (query, head): M = max m_c, w_c = 2^(m_c - M), L = sum l_c w_c, out = sum
// acc_c w_c / L, c over the runs (the raw tail's is the last).
//
// Rows of at most 32 runs: a warp per head and 64 dims, eight a CTA.  Longer ones: a
// CTA per head.  Both add in the same order -- eight sums over the runs c = s,
// s+8, .. (s < 8), added in order of s -- so that a row's bits do not depend on
// which of the two its batch takes.  Latency bound (2.1 us for 8 rows of 8 runs,
// 6.8 us for 8 rows of 256): every load that can be is made before the first is
// used.  Launching it early, to wait resident beside the runs' CTAs, took 2-5 us
// more than its launch saved.
constexpr int kMergeThreads = 256;
constexpr int kMergeWarps = kMergeThreads / 32;
constexpr int kSlices = 8;
constexpr int kWarpRuns = 32;
constexpr int kMaxRuns = 513;
constexpr int kRunsPerThread = (kMaxRuns + kMergeThreads - 1) / kMergeThreads;

template <int D>
using Vec = typename std::conditional<D == 128, float4, float2>::type;  // a lane's dims
template <typename V>
__device__ __forceinline__ float at(const V &v, int j) { return reinterpret_cast<const float *>(&v)[j]; }
template <typename V>
__device__ __forceinline__ float &at(V &v, int j) { return reinterpret_cast<float *>(&v)[j]; }

__device__ __forceinline__ int used_runs(const AttendCodedArgs &a, const Row &row)
{
    return coded_runs(row.groups, a.ids == nullptr, a.q_heads / a.kv_heads) + (row.tail > 0 ? 1 : 0);
}

__device__ __forceinline__ float inverse(float L)  // of a denominator; 0: no token (or none above -inf)
{
    return L > 0.0f || L != L ? 1.0f / L : 0.0f;
}

// Unit u: 64 dims of head u / (D/64), two a lane.  The states are loaded before the row's
// length is known: `most` bounds the runs of the call's rows, and what is behind this
// row's runs is not used.
template <int D>
__device__ __forceinline__ void merge_by_warp(const AttendCodedArgs &a, int b, int u, int most)
{
    constexpr int kHalves = D / 64;
    constexpr int kNext = 4;
    const int h = u / kHalves, col = (u % kHalves) * 32 + (threadIdx.x & 31);
    const int lane = threadIdx.x & 31;
    const int64_t hb = int64_t(b) * a.q_heads + h;
    const float2 *src = reinterpret_cast<const float2 *>(a.part_acc + hb * a.nparts * D) + col;
    float pm = -INFINITY, pl = 0.0f;
    if (lane < most) {
        pm = __ldcg(a.part_m + hb * a.nparts + lane);
        pl = __ldcg(a.part_l + hb * a.nparts + lane);
    }
    float2 sum[kSlices], next[kNext];
#pragma unroll
    for (int s = 0; s < kSlices; ++s)
        if (s < most) sum[s] = __ldcg(src + int64_t(s) * (D / 2));
#pragma unroll
    for (int k = 0; k < kNext; ++k)
        if (kSlices + k < most) next[k] = __ldcg(src + int64_t(kSlices + k) * (D / 2));
    const int used = used_runs(a, row_of(a, b));
    if (lane >= used) pm = -INFINITY;
    float m = pm;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float M = m == -INFINITY ? 0.0f : m;
    const float w = lane < used ? ex2(pm - M) : 0.0f;
    float L = lane < used ? fmaf(pl, w, 0.0f) : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
#pragma unroll
    for (int s = 0; s < kSlices; ++s) {
        const float ws = __shfl_sync(0xffffffffu, w, s);
        sum[s] = s < used ? make_float2(fmaf(sum[s].x, ws, 0.0f), fmaf(sum[s].y, ws, 0.0f)) : make_float2(0.0f, 0.0f);
    }
    for (int c0 = kSlices; c0 < used; c0 += kSlices) {
#pragma unroll
        for (int s0 = 0; s0 < kSlices; s0 += kNext) {
#pragma unroll
            for (int k = 0; k < kNext; ++k) {
                const int c = c0 + s0 + k;
                const float ws = __shfl_sync(0xffffffffu, w, c & 31);
                if (c < used) sum[s0 + k] = make_float2(fmaf(next[k].x, ws, sum[s0 + k].x), fmaf(next[k].y, ws, sum[s0 + k].y));
                if (c + kNext < used) next[k] = __ldcg(src + int64_t(c + kNext) * (D / 2));
            }
        }
    }
    float2 out = sum[0];
#pragma unroll
    for (int s = 1; s < kSlices; ++s) out = make_float2(out.x + sum[s].x, out.y + sum[s].y);
    out = L > 0.0f || L != L ? make_float2(out.x / L, out.y / L) : make_float2(0.0f, 0.0f);
    reinterpret_cast<float2 *>(a.out + hb * D)[col] = out;
    if (a.stat != nullptr && col == 0) reinterpret_cast<float2 *>(a.stat)[hb] = make_float2(M, inverse(L));
}

template <int D>
__device__ __forceinline__ void merge_by_block(const AttendCodedArgs &a, int b, int h, const Row &row)
{
    constexpr int kPer = D / 32;
    constexpr int kAhead = 8;
    __shared__ float w[kMaxRuns];
    __shared__ float red[2][kMergeWarps];
    __shared__ Vec<D> part[kSlices][32];
    static_assert(kMergeWarps == kSlices, "a warp per slice");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int used = used_runs(a, row);
    const int64_t hb = int64_t(b) * a.q_heads + h;
    const Vec<D> *src = reinterpret_cast<const Vec<D> *>(a.part_acc + hb * a.nparts * D) + lane;
    float pm[kRunsPerThread], pl[kRunsPerThread];
#pragma unroll
    for (int k = 0; k < kRunsPerThread; ++k) {
        const int c = tid + k * kMergeThreads;
        pm[k] = c < used ? __ldcg(a.part_m + hb * a.nparts + c) : -INFINITY;
        pl[k] = c < used ? __ldcg(a.part_l + hb * a.nparts + c) : 0.0f;
    }
    Vec<D> x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
        if (warp + u * kSlices < used) x[u] = __ldcg(src + int64_t(warp + u * kSlices) * 32);
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < kRunsPerThread; ++k) m = fmaxf(m, pm[k]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) red[0][warp] = m;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMergeWarps; ++k) m = fmaxf(m, red[0][k]);
    const float M = m == -INFINITY ? 0.0f : m;
    float l = 0.0f;
#pragma unroll
    for (int k = 0; k < kRunsPerThread; ++k) {
        const int c = tid + k * kMergeThreads;
        if (c >= used) continue;
        w[c] = ex2(pm[k] - M);
        l = fmaf(pl[k], w[c], l);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) red[1][warp] = l;
    __syncthreads();
    float L = red[1][0];
#pragma unroll
    for (int k = 1; k < kMergeWarps; ++k) L += red[1][k];
    float o[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) o[j] = 0.0f;
    for (int c0 = warp; c0 < used; c0 += kAhead * kSlices) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int c = c0 + u * kSlices;
            if (c < used) {
#pragma unroll
                for (int j = 0; j < kPer; ++j) o[j] = fmaf(at(x[u], j), w[c], o[j]);
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int c = c0 + (kAhead + u) * kSlices;
            if (c < used) x[u] = __ldcg(src + int64_t(c) * 32);
        }
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) at(part[warp][lane], j) = o[j];
    __syncthreads();
    if (warp != 0) return;
    Vec<D> out;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        float y = o[j];
#pragma unroll
        for (int s = 1; s < kSlices; ++s) y += at(part[s][lane], j);
        at(out, j) = L > 0.0f || L != L ? y / L : 0.0f;
    }
    reinterpret_cast<Vec<D> *>(a.out + hb * D)[lane] = out;
    if (a.stat != nullptr && lane == 0) reinterpret_cast<float2 *>(a.stat)[hb] = make_float2(M, inverse(L));
}

// ---- the groups' shares of attention ------------------------------------------------------
// weights[weight_offset[b] + g] += sum_h share(b, h, g), share = mass * 2^(mref - M_h) / L_h.
// No atomics: a query with accumulators of its own adds its shares as they come
// (own_weights, CTAs beside the merge's, which find M and L themselves from the
// runs' states rather than wait for the merge); queries that share accumulators
// are added in a fixed order, up to 32 partial sums per group (shared_weights_kernel), so
// that the sum has one value.  Selected rows of such queries are first spread out
// to one share per group of the history (in the workspace's scores, which nobody
// needs by then), so that the second kernel reads rows side by side: on 256
// queries that share a history of 25,064 groups, searching each group in each
// query's row instead took 1540 us, this 14 us.
constexpr int kAccThreads = kMergeThreads;
constexpr int kOwnPos = kAccThreads;                   // positions of a CTA, one per thread
constexpr int kStatHeads = 64;                         // heads whose M and 1/L are in hand at a time
constexpr int kSharedGroups = 32;                      // groups of a unit of work
constexpr int kManySlices = 32, kFewSlices = 8;        // parts of a sum over queries: of more than eight, of up to eight
constexpr int kList = 512;                             // queries of a history in hand at a time
constexpr int kSharedCtas = 608;                       // 4 per SM; the sums do not depend on it

// M and 1/L of a head from its runs' states, by a warp.
__device__ __forceinline__ float2 stat_of_runs(const AttendCodedArgs &a, int64_t hb, int used)
{
    const float *pm = a.part_m + hb * a.nparts, *pl = a.part_l + hb * a.nparts;
    float m = -INFINITY, l = 0.0f;
#pragma unroll 4
    for (int c = threadIdx.x & 31; c < used; c += 32) {
        const float mc = __ldcg(pm + c), lc = __ldcg(pl + c);
        const float mn = fmaxf(m, mc);
        const float ms = mn == -INFINITY ? 0.0f : mn;
        l = fmaf(l, ex2(m - ms), lc * ex2(mc - ms));
        m = mn;
    }
    float M = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (M == -INFINITY) M = 0.0f;
    l *= ex2(m - M);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    return make_float2(M, inverse(l));
}

// CTA `x` of `n` for query b.
__device__ __forceinline__ void own_weights(const AttendCodedArgs &a, int b, int x, int n, const Row &row)
{
    __shared__ float2 stat[kStatHeads];
    const int tid = threadIdx.x, warp = tid >> 5;
    const bool whole = a.ids == nullptr;
    const uint32_t sharing = __ldcg(a.sharing + b);
    const bool own = sharing == 0;
    // (shared accumulators of whole histories: shared_weights_kernel reads the masses itself)
    const int first = !own && whole ? row.groups : 0, end = row.groups + (row.tail > 0 ? 1 : 0);
    if ((sharing & kBad) || first + int64_t(x) * kOwnPos >= end) return;
    const int used = used_runs(a, row);
    const int64_t hb0 = int64_t(b) * a.q_heads;
    for (int64_t p0 = first + int64_t(x) * kOwnPos; p0 < end; p0 += int64_t(n) * kOwnPos) {
        const int p = int(p0) + tid;
        int g = row.T / kGroup;
        if (p < row.groups) g = whole ? p : __ldcg(a.ids + int64_t(b) * a.row_cap + kGroup * int64_t(p)) / kGroup;
        float s = 0.0f;
        for (int h0 = 0; h0 < a.q_heads; h0 += kStatHeads) {
            const int nh = min(kStatHeads, a.q_heads - h0);
            if (p0 == first + int64_t(x) * kOwnPos || a.q_heads > kStatHeads) {
                __syncthreads();
#pragma unroll 2
                for (int h = warp; h < nh; h += kMergeWarps) {
                    const float2 st = stat_of_runs(a, hb0 + h0 + h, used);
                    if (tid % 32 == 0) stat[h] = st;
                }
                __syncthreads();
            }
            if (p >= end) continue;
            const float *mass = a.mass + (hb0 + h0) * a.mass_stride + p;
            const float *mref = a.mref + (hb0 + h0) * (a.mass_stride / 4) + p / 4;
            int64_t ms = a.mass_stride, rs = a.mass_stride / 4;
            if (p == row.groups) {  // the raw tail: its run's state
                mass = a.part_l + (hb0 + h0) * a.nparts + used - 1;
                mref = a.part_m + (hb0 + h0) * a.nparts + used - 1;
                ms = rs = a.nparts;
            }
#pragma unroll 8
            for (int h = 0; h < nh; ++h)
                s = fmaf(__ldcg(mass + h * ms) * ex2(__ldcg(mref + h * rs) - stat[h].x), stat[h].y, s);
        }
        if (p >= end) continue;
        if (own) a.weights[__ldg(a.weight_offset + b) + g] += s;
        else if (p == row.groups) a.tail_share[b] = s;
        else a.share_map[int64_t(b) * a.map_stride + g] = s;
    }
}

// CTAs per SM: without the weights' code there are registers for five (1,024 queries of
// two runs, 16 heads x 128: 13.5 -> 12.1 us; six take 11.7, but 12 queries of 18 runs
// 4.7 instead of 3.4, too few of their loads being under way at a time).
template <int D, bool kByWarp, bool kOwn>
__global__ void __launch_bounds__(kMergeThreads, kByWarp && !kOwn ? 5 : 4)
merge_coded_kernel(const AttendCodedArgs a, int merge_ctas, int most)
{
    const int x = blockIdx.x, b = blockIdx.y;
    wait_for_predecessor();
    if (kOwn && x >= merge_ctas) {
        if constexpr (kOwn) own_weights(a, b, x - merge_ctas, int(gridDim.x) - merge_ctas, row_of(a, b));
    } else if constexpr (kByWarp) {
        const int u = x * kMergeWarps + (threadIdx.x >> 5);
        if (u < a.q_heads * (D / 64)) merge_by_warp<D>(a, b, u, most);
    } else {
        merge_by_block<D>(a, b, x, row_of(a, b));
    }
}

// Groups g .. g+3 of a whole history, whose masses have one reference.
__device__ __forceinline__ float4 shares_of(const AttendCodedArgs &a, int b, int g)
{
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int64_t hb = int64_t(b) * a.q_heads, step = a.mass_stride / 4;
    const float4 *mass = reinterpret_cast<const float4 *>(a.mass + hb * a.mass_stride + g);
    const float *mref = a.mref + hb * step + g / 4;
    const float2 *stat = reinterpret_cast<const float2 *>(a.stat) + hb;
#pragma unroll 4
    for (int h = 0; h < a.q_heads; ++h) {
        const float4 m = __ldcg(mass + h * step);
        const float2 st = __ldcg(stat + h);
        const float e = ex2(__ldcg(mref + h * step) - st.x);
        s.x = fmaf(m.x * e, st.y, s.x);
        s.y = fmaf(m.y * e, st.y, s.y);
        s.z = fmaf(m.z * e, st.y, s.z);
        s.w = fmaf(m.w * e, st.y, s.w);
    }
    return s;
}

// The work is cut into units of kSharedGroups groups of one history, and the units
// dealt out in contiguous shares, so that a CTA lists a history's queries once for
// all the groups that it takes of it.  The list leaves out the batch's other queries:
// a sum depends on the queries of its history alone.  It holds kList queries; those
// of a larger history are added a list at a time.  64 histories of 2,048
// groups and 4 queries each: 8.2 us for selected rows, 19 us for whole ones (four CTAs
// per SM, four groups a thread; one group a thread 7.7 and 26, and 16 instead of 14 on
// 256 queries of one history; with six CTAs 9.7 and 72: too few registers for the loads
// in flight); with a block of groups per CTA and a pass over the whole batch for each
// history 222 and 482.
template <bool kWhole>
__global__ void __launch_bounds__(kAccThreads, 4) shared_weights_kernel(const AttendCodedArgs a)
{
    __shared__ int2 list[kList + kAccThreads];  // a query, and 2 * its history's groups + (it has a raw tail)
    __shared__ float4 sum[kAccThreads];
    __shared__ uint32_t marked[kAccThreads / 32];
    __shared__ int found;
    constexpr int kAhead = 4;                   // loads made before the first is added
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int groups = a.max_visible / kGroup + 1;
    const int per_history = (groups + kSharedGroups - 1) / kSharedGroups;
    wait_for_predecessor();

    // marks the threads that pass true: the marked ones before this one, and all of them
    auto mark = [&](bool x, int &total) {
        const uint32_t votes = __ballot_sync(0xffffffffu, x);
        __syncthreads();
        if (lane == 0) marked[warp] = votes;
        __syncthreads();
        int before = __popc(votes & ((1u << lane) - 1u));
        total = 0;
#pragma unroll
        for (int w = 0; w < kAccThreads / 32; ++w) {
            if (w < warp) before += __popc(marked[w]);
            total += __popc(marked[w]);
        }
        return before;
    };
    // blocks blk0 .. blk1 of the history of `off`: the first n queries of the list added, in
    // `slices` sums over the queries k, k + slices, .. that are added in order of k.  (Up
    // to eight queries are one to a sum either way.)
    auto add_list = [&](int64_t off, int blk0, int blk1, int n) {
        const int slices = n <= kFewSlices ? kFewSlices : kManySlices, quads = kAccThreads / slices;
        const int slice = tid / quads, quad = tid % quads;
        const int end = min(blk1 * kSharedGroups, groups);
        for (int g0 = blk0 * kSharedGroups; g0 < end; g0 += 4 * quads) {
            const int g = g0 + 4 * quad;
            float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            auto add = [&](const float4 &t, int history) {
                s.x += g < history ? t.x : 0.0f;
                s.y += g + 1 < history ? t.y : 0.0f;
                s.z += g + 2 < history ? t.z : 0.0f;
                s.w += g + 3 < history ? t.w : 0.0f;
            };
            if (g < end) {
                if constexpr (kWhole) {
                    for (int j = slice; j < n; j += slices)
                        if (g < list[j].y / 2) add(shares_of(a, list[j].x, g), list[j].y / 2);
                } else {
                    const float *map = a.share_map + min(g, a.map_stride - 4);
                    for (int j = slice; j < n; j += slices * kAhead) {
                        float4 t[kAhead];
#pragma unroll
                        for (int u = 0; u < kAhead; ++u)  // (every load is made, no branch between them)
                            t[u] = __ldcg(reinterpret_cast<const float4 *>(map + int64_t(list[min(j + u * slices, n - 1)].x) * a.map_stride));
#pragma unroll
                        for (int u = 0; u < kAhead; ++u)
                            if (j + u * slices < n) add(t[u], list[j + u * slices].y / 2);
                    }
                }
                for (int j = slice; j < n; j += slices) {  // the raw tails
                    const int2 m = list[j];
                    if ((m.y & 1) && (m.y / 2 & ~3) == g) {
                        const float t = __ldcg(a.tail_share + m.x);
                        const int at = m.y / 2 - g;
                        s.x += at == 0 ? t : 0.0f;
                        s.y += at == 1 ? t : 0.0f;
                        s.z += at == 2 ? t : 0.0f;
                        s.w += at == 3 ? t : 0.0f;
                    }
                }
            }
            sum[tid] = s;  // [slices][quads]
            __syncthreads();
            if (tid < 4 * quads && g0 + tid < end) {
                const float *part = reinterpret_cast<const float *>(sum) + tid;
                float w = part[0];
                for (int k = 1; k < min(n, slices); ++k) w += part[k * 4 * quads];
                if (w != 0.0f) a.weights[off + g0 + tid] += w;
            }
            __syncthreads();
        }
    };

    // the histories that queries share, by their first queries
    auto is_first = [&](int b) { return b < a.batch && (__ldcg(a.sharing + b) & kFirstSharer); };
    int histories = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kAccThreads) histories += __syncthreads_count(is_first(b0 + tid));
    const int64_t units = int64_t(histories) * per_history;
    const int64_t end = units * (blockIdx.x + 1) / gridDim.x;
    int64_t unit = units * blockIdx.x / gridDim.x;
    int b0 = 0, passed = 0;                     // first queries before b0
    while (unit < end) {
        const int nth = int(unit / per_history), blk0 = int(unit - int64_t(nth) * per_history);
        const int blk1 = int(min(int64_t(per_history), blk0 + (end - unit)));
        unit += blk1 - blk0;
        for (int total;; b0 += kAccThreads, passed += total) {
            const bool first = is_first(b0 + tid);
            const int before = mark(first, total);
            if (first && passed + before == nth) found = b0 + tid;
            if (nth < passed + total) break;
        }
        __syncthreads();
        const int64_t off = __ldg(a.weight_offset + found);
        int n = 0;
        for (int o0 = found; o0 < a.batch; o0 += kAccThreads) {
            const int o = o0 + tid;
            const bool member = o < a.batch && __ldg(a.weight_offset + o) == off && !(__ldcg(a.sharing + o) & kBad);
            int total;
            const int at = n + mark(member, total);
            if (member) {
                const Row row = row_of(a, o);
                list[at] = make_int2(o, row.T / kGroup * 2 + (row.tail > 0 ? 1 : 0));
            }
            n += total;
            __syncthreads();
            const bool last = o0 + kAccThreads >= a.batch;
            while (n >= kList || (last && n > 0)) {
                const int taken = min(n, kList);
                add_list(off, blk0, blk1, taken);
                __syncthreads();
                const int2 rest = list[taken + min(tid, kAccThreads - 1)];  // at most kAccThreads - 1 are left
                __syncthreads();
                n -= taken;
                if (tid < n) list[tid] = rest;
                __syncthreads();
            }
        }
    }
}

template <int D, bool kOwn>
cudaError_t launch_merge_t(const AttendCodedArgs &a, cudaStream_t s)
{
    int own = 0;
    if (kOwn) {
        const int positions = (a.ids == nullptr ? a.max_visible : a.row_cap) / kGroup + 1;
        own = (positions + kOwnPos - 1) / kOwnPos;
        if (own > 1024) own = 1024;
    }
    const bool whole = a.ids == nullptr;
    const int most = whole ? a.nparts : coded_runs((a.row_cap - (kGroup - 1)) / kGroup, false, a.q_heads / a.kv_heads) + 1;
    const bool by_warp = most <= kWarpRuns;
    const int ctas = by_warp ? (a.q_heads * (D / 64) + kMergeWarps - 1) / kMergeWarps : a.q_heads;
    return launch_kernel(by_warp ? merge_coded_kernel<D, true, kOwn> : merge_coded_kernel<D, false, kOwn>,
                         dim3(unsigned(ctas + own), unsigned(a.batch)), dim3(kMergeThreads), 0, s, true, a, ctas, most);
}

}  // namespace

cudaError_t launch_merge_coded(const AttendCodedArgs &a, cudaStream_t s)
{
    const bool own = a.weights != nullptr;
    const cudaError_t e = a.head_dim == 128 ? (own ? launch_merge_t<128, true>(a, s) : launch_merge_t<128, false>(a, s))
                                            : (own ? launch_merge_t<64, true>(a, s) : launch_merge_t<64, false>(a, s));
    if (e != cudaSuccess || !own || a.batch == 1) return e;
    const int64_t most = int64_t(a.max_visible / kGroup + kSharedGroups) / kSharedGroups * (a.batch / 2);  // units
    return launch_kernel(a.ids == nullptr ? shared_weights_kernel<true> : shared_weights_kernel<false>,
                         dim3(unsigned(most < kSharedCtas ? most : kSharedCtas)), dim3(kAccThreads), 0, s, true, a);
}

}  // namespace qsa
