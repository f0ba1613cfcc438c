// attend_coded4.cu -- attention of one query per batch entry over K/V rows held in 4-bit
// codes with a scale per 4 x 4 tile and one per (group, KV head) (include/qsa_cache.h:
// qsa_attend_coded), with the attention that each group received.
//
// The mathematics and the shape are those of attend_coded.cu: m16n8k16 products of q and of the
// weights, each as hi + lo of two 16-bit floats, with codes that are exact in one -- here a code
// times its tile's scale t, at most 7 significant bits -- and the group's scale applied to the
// result (K) or to the weight (V).  What differs:
//
// Decoding.  Two codes become an operand register by one conversion (e2m1) or one masking into
// the low bits of 1024 or 64 (int4), and one multiplication by t.  The layout has the two codes
// of a pair where that finds them, a lane's codes side by side, and a tile in one lane.
//
// Steps of 8 groups (32 tokens).  Half the bytes per group halve the time that a step's fixed work
// may take, so two products' tokens share a step's softmax, power of two and sums of values, and
// q's operands are read from shared memory once for both (registers hold none of them).  No
// lane compares its scores with the other lanes' until one passes the reference by 2^kLag.
// (Steps of 4 groups with q in registers: 8 histories of 262,144 tokens 164 us instead of 153
// at that time.)
//
// Bound: by the latency of a warp's own chain (copy wait, shared loads, decoding, dependent products, softmax with two
// shuffles, split, products), four warps to a scheduler, not by memory and not by a pipe.  8 histories of 262,144 tokens (16 / 2
// heads x 128, e2m1, 612 MB, 92 us at the copy rate): 138.5 us a call, 10 of it merge and
// launches; from a cache that fits L2 it takes 133, without both products 111, and with
// neither 55.  16 tokens cost a warp 64 conversions, 64 half multiplications and 32 matrix
// instructions, which alone take 335-355 cycles of a scheduler (mma.sync 256 of them: it does 256
// products a cycle here), and some 190 others; the kernel takes 618, with half of the issue slots and 36 % of the
// tensor pipe used, and 11 instructions a step less measured the same.  Nothing here starts the scores of the next
// step before the values of this one.  int4 150 us: its decoding takes 9 instructions a word and 3
// per tile pair for the offsets, against 8 and none.  32 ragged rows of up to 65,537 tokens, int4: 76.
// 9 to 16 heads: twice the matrix instructions for the same codes (4 x 40,003 tokens of 16 heads
// on one, with weights: 29, three quarters of a wave of runs).
// Tried and not kept: a ring of three at three CTAs per SM (166 us), five CTAs with 96
// registers (162), runs twice as long for 4 bits (no faster for the longest rows, 83 -> 92 for
// ragged ones), 128 groups resolved at a time, heads as the slower dimension of the grid (the
// two heads of a block read far apart: 7 us more).
#include "attend_coded_common.cuh"
#include "codes4.cuh"

namespace qsa {
namespace {

constexpr int kSubGroups = 4;                   // groups of a product's 16 tokens
constexpr int kSub = 2;                         // products whose softmax and whose sums of values are taken together: a warp step
constexpr int kStepGroups = kSub * kSubGroups;
constexpr int kRing = 2;                        // a warp's steps in shared memory: one in use, one on its way
constexpr int kSegGroups = 256;                 // groups resolved at a time
constexpr int kEach = kSegGroups / kThreads;    // .. by a thread

template <int D, int HS, int F>
struct Sm {
    // a block and, behind it, the bytes that keep the reads of both products free of conflicts
    static constexpr int kBlk = code_bytes(F, D) + (D == 64 ? 0 : 32);
    static constexpr int kStage = kStepGroups * kBlk;
    alignas(128) unsigned char ring[kWarps][kRing][kStage];  // also the end-of-run reduction area
    alignas(16) float4 meta[kSegGroups];                     // K scale, V scale and its exponent, 0 (-inf: no such group)
    alignas(16) uint4 qa[D / 16][HS][32];                    // each lane's operands of q (9-16 heads: hi, lo)
    float qs[8 * HS];                                        // 1/f of each head's q
    alignas(16) int blk[kSegGroups];                         // physical block; -1: none, -2: zero rows
    float wm[kWarps][8 * HS], wl[kWarps][8 * HS];
};

// CTAs per SM that the registers and the ring leave room for.
template <int D, int HS>
constexpr int ctas_per_sm() { return HS == 2 ? 3 : D == 128 ? 4 : 6; }

template <int D, int HS, int F>
__global__ void __launch_bounds__(kThreads, (ctas_per_sm<D, HS>())) attend_coded4_kernel(const AttendCodedArgs a)
{
    extern __shared__ __align__(128) unsigned char smem_raw[];
    using S = Sm<D, HS, F>;
    S &sm = *reinterpret_cast<S *>(smem_raw);
    constexpr int kBytes = code_bytes(F, D);
    constexpr int kNH = 8 * HS;
    constexpr int kHalves = D / 64;       // 64-dim halves of K
    constexpr int kVC = D / 32;           // 16-byte V reads per lane and group
    constexpr int kChains = HS;  // independent accumulations of a score tile

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int hl = lane >> 2, i4 = lane & 3;
    const int gq = a.q_heads / a.kv_heads;
    const bool whole = a.ids == nullptr;

    wait_for_predecessor();
    // the first CTAs of each (query, KV head): the raw tail, and what belongs to the query as a whole
    const int extra = a.sharing != nullptr ? 2 : 1;
    const int part = int(blockIdx.x) / a.kv_heads - extra, kvh = int(blockIdx.x) % a.kv_heads, b = blockIdx.z;
    const int h0 = kvh * gq;
    if (part == -2 && kvh != 0) return;
    const int64_t block_offset = __ldg(a.block_offset + b);  // (under way while the row is looked up)
    const Row row = row_of(a, b);
    if (part < 0) {
        if (part == -2) {
            find_sharing(a, b, row);
            return;
        }
        if (kvh == 0 && tid == 0) {
            if (a.n_ids_out != nullptr) a.n_ids_out[b] = __ldcg(a.n_ids + b);
            if (!row.ok) set_error(a.err, row.t_ok ? QSA_DEVERR_ROW_RANGE : QSA_DEVERR_VISIBLE_RANGE);
        }
        if (row.tail > 0) attend_tail<D>(a, b, kvh, row, coded_runs(row.groups, whole, gq));
        return;
    }
    if (a.share_map != nullptr && !whole) {  // the query's row of shares cleared, a slice by each of its CTAs
        const int ctas = int(gridDim.x) - extra * a.kv_heads, n = (a.map_stride / 4 + ctas - 1) / ctas;
        const int g0 = (part * a.kv_heads + kvh) * n;
        float4 *map = reinterpret_cast<float4 *>(a.share_map + int64_t(b) * a.map_stride);
        for (int g = g0 + tid; g < min(g0 + n, a.map_stride / 4); g += kThreads) map[g] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int per_run = coded_run_groups(row.groups, whole, gq);
    const int run_begin = part * per_run, run_end = min(row.groups, run_begin + per_run);
    if (run_begin >= run_end) return;

    // A run is taken in segments of up to kSegGroups groups, thread t resolving groups
    // seg + t, ..: its block first, so that copies can start, ...
    auto load_block = [&](int g) {
        if (g >= run_end) return -1;
        if (!whole) {
            const int64_t at = int64_t(b) * a.row_cap + kGroup * int64_t(g);
            int id[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) id[u] = __ldcg(a.ids + at + u);
            if (kvh == 0 && a.ids_out != nullptr) {
#pragma unroll
                for (int u = 0; u < 4; ++u) a.ids_out[at + u] = id[u];
            }
            g = id[0] / kGroup;
            if (!(id[0] >= 0 && id[0] % kGroup == 0 && id[0] <= row.T - kGroup && id[1] == id[0] + 1 && id[2] == id[0] + 2 &&
                  id[3] == id[0] + 3)) {
                set_error(a.err, QSA_DEVERR_ROW_RANGE);
                return -2;
            }
        }
        const int blk = __ldg(a.block_map + block_offset + g);
        if (blk < 0 || blk >= a.num_blocks) {
            set_error(a.err, QSA_DEVERR_SLOT_RANGE);
            return -2;
        }
        return blk;
    };
    // ... then its scales
    auto load_scales = [&](int blk) {
        return blk >= 0 ? __ldg(reinterpret_cast<const float2 *>(a.scales) + int64_t(blk) * a.kv_heads + kvh)
                        : make_float2(0.0f, 0.0f);
    };
    auto store_meta = [&](int at, int blk, float2 sc) {
        const uint32_t bits = __float_as_uint(sc.y) & 0x7fffffffu;
        const float e = bits == 0 ? -INFINITY : float(int(bits >> 23) - 127);
        sm.meta[at] = make_float4(sc.x, sc.y, e, blk != -1 ? 0.0f : -INFINITY);
    };
    const unsigned char *codes = a.codes + int64_t(kvh) * kBytes + lane * 16;  // this lane's first piece of block 0
    const uint32_t blk_bytes = uint32_t(a.kv_heads) * kBytes;
    auto at_block = [&](int blk) { return codes + uint64_t(uint32_t(blk)) * blk_bytes; };  // one instruction
    const uint32_t ring = smem_u32(sm.ring[warp]) + lane * 16;
    auto issue = [&](int g0, uint32_t slot) {  // the step at group g0 of the segment, into ring bytes slot
        int blk[kStepGroups], least = 0;
#pragma unroll
        for (int v = 0; v < kSub; ++v) {
            const int4 b4 = *reinterpret_cast<const int4 *>(sm.blk + g0 + kSubGroups * v);
            blk[4 * v] = b4.x, blk[4 * v + 1] = b4.y, blk[4 * v + 2] = b4.z, blk[4 * v + 3] = b4.w;
            least = min(least, min(min(b4.x, b4.y), min(b4.z, b4.w)));
        }
        if (least >= 0) {
            if constexpr (D == 128) {  // a block's codes are a piece per lane, its tile scales four more
#pragma unroll
                for (int u = 0; u < kStepGroups; ++u) cp_async16(ring + slot + u * S::kBlk, at_block(blk[u]));
                if (lane < 4 * kStepGroups) {
                    const int u = lane / 4, to = 4 * D - 64 * u;  // (lane * 16 is 64 u + 16 (lane%4))
                    cp_async16(ring + slot + u * S::kBlk + to, at_block(sm.blk[g0 + u]) + to);
                }
            } else {                   // 16 pieces of codes, two of tile scales
                const int half = lane / 16;
#pragma unroll
                for (int v = 0; v < kStepGroups / 2; ++v) {
                    const int u = 2 * v + half, to = -256 * half;
                    cp_async16(ring + slot + u * S::kBlk + to, at_block(half ? blk[2 * v + 1] : blk[2 * v]) + to);
                }
                if (lane < 2 * kStepGroups) {
                    const int u = lane / 2, to = 4 * D - 32 * u;
                    cp_async16(ring + slot + u * S::kBlk + to, at_block(sm.blk[g0 + u]) + to);
                }
            }
        } else {  // some groups are not there, or not to be read: zeros
            for (int u = 0; u < kStepGroups; ++u) {
                const int bu = sm.blk[g0 + u];
                for (int c = 0; c < kBytes; c += 512) {
                    if (c + lane * 16 >= kBytes) break;
                    if (bu >= 0) cp_async16(ring + slot + u * S::kBlk + c, at_block(bu) + c);
                    else *reinterpret_cast<uint4 *>(&sm.ring[warp][0][0] + slot + u * S::kBlk + c + lane * 16) = make_uint4(0, 0, 0, 0);
                }
            }
        }
        cp_async_commit();
    };
    // this warp's steps of a segment: groups kStepGroups * (warp + kWarps * k)
    auto steps_of = [&](int seg) {
        const int n = (min(kSegGroups, run_end - seg) + kStepGroups - 1) / kStepGroups;
        return n > warp ? (n - warp + kWarps - 1) / kWarps : 0;
    };
    auto first_steps = [&](int my_steps) {
#pragma unroll
        for (int k = 0; k < kRing - 1; ++k) {
            if (k < my_steps) issue((warp + kWarps * k) * kStepGroups, k * S::kStage);
            else cp_async_commit();
        }
    };

    int my_blk[kEach];
    float2 my_scales[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) my_blk[e] = load_block(run_begin + tid + kThreads * e);
#pragma unroll
    for (int e = 0; e < kEach; ++e) sm.blk[tid + kThreads * e] = my_blk[e];
    __syncthreads();
    int my_steps = steps_of(run_begin);
    first_steps(my_steps);
#pragma unroll
    for (int e = 0; e < kEach; ++e) my_scales[e] = load_scales(my_blk[e]);

    // ---- the queries: 16 threads a head, each 8 dims at a time, to the matrix operands -----
    // of the lane that holds the dims: words u of dims 8(u/2) + 2(u%2) + 0, 4, 1, 5
    // of 64j + 16*i4, hi and lo, with the head's power of two taken out
    constexpr int kQPer = D / 128 > 0 ? D / 128 : 1;   // pieces of 8 dims per thread and head
    constexpr int kQThreads = D / 8 / kQPer;           // threads per head: 16, or 8 for d = 64
#pragma unroll
    for (int h0q = 0; h0q < 8 * HS; h0q += kThreads / kQThreads) {
        const int h = h0q + tid / kQThreads, c = tid % kQThreads;  // dims 8c..8c+7
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        if (h < gq) {
            const float4 *src = reinterpret_cast<const float4 *>(a.q + (int64_t(b) * a.q_heads + h0 + h) * D) + 2 * c;
            x = __ldg(src);
            y = __ldg(src + 1);
        }
        uint32_t top = 0;
        for (const float v : {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w}) top = max(top, __float_as_uint(v) & 0x7fffffffu);
#pragma unroll
        for (int o = 1; o < kQThreads; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        float f, inv;
        scale_of_q(top, f, inv);
        if (h >= 8 * HS) continue;  // (d = 64: more threads than heads need)
        uint32_t hi[4], lo[4];
        // the pairs of a word: dims p and p + 4
        split2(make_float2(x.x * f, y.x * f), hi[0], lo[0]);
        split2(make_float2(x.y * f, y.y * f), hi[1], lo[1]);
        split2(make_float2(x.z * f, y.z * f), hi[2], lo[2]);
        split2(make_float2(x.w * f, y.w * f), hi[3], lo[3]);
        const int e = 4 * (c / 8) + 2 * (c % 2), to = (h % 8) * 4 + (c % 8) / 2;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if constexpr (HS == 1) {
                sm.qa[e + u][0][to] = make_uint4(hi[2 * u], lo[2 * u], hi[2 * u + 1], lo[2 * u + 1]);
            } else {  // rows hl and hl + 8 of an operand are heads: the second set's words are y and w
                uint32_t *const ph = reinterpret_cast<uint32_t *>(&sm.qa[e + u][0][to]) + h / 8;
                uint32_t *const pl = reinterpret_cast<uint32_t *>(&sm.qa[e + u][HS - 1][to]) + h / 8;
                ph[0] = hi[2 * u], ph[2] = hi[2 * u + 1];
                pl[0] = lo[2 * u], pl[2] = lo[2 * u + 1];
            }
        }
        if (c == 0) sm.qs[h] = inv;
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) store_meta(tid + kThreads * e, my_blk[e], my_scales[e]);
    __syncthreads();
    const Int4Base int4_base(uint32_t(a.batch >> 31));
    float hscale[HS];
#pragma unroll
    for (int s = 0; s < HS; ++s) hscale[s] = a.scale * kLog2e * sm.qs[hl + 8 * s] * kUnits<F>;

    // the accumulator: dims 32*j + 8*i4 + u (x) and + 4 (y) of head hl + 8*s
    float2 acc[HS][kVC][4];
    float m_run[HS], l_run[HS];
    float mref[HS], m_pass[HS];  // what scores are taken relative to (m_run, or 0 while that is -inf); what none may pass
#pragma unroll
    for (int s = 0; s < HS; ++s) {
        m_run[s] = m_pass[s] = -INFINITY;
        l_run[s] = mref[s] = 0.0f;
#pragma unroll
        for (int j = 0; j < kVC; ++j)
#pragma unroll
            for (int u = 0; u < 4; ++u) acc[s][j][u] = make_float2(0.0f, 0.0f);
    }

    for (int seg = run_begin; seg < run_end; seg += kSegGroups) {
        if (seg != run_begin) {  // every warp is done with the last segment's blocks
            __syncthreads();
#pragma unroll
            for (int e = 0; e < kEach; ++e) my_blk[e] = load_block(seg + tid + kThreads * e);
#pragma unroll
            for (int e = 0; e < kEach; ++e) sm.blk[tid + kThreads * e] = my_blk[e];
#pragma unroll
            for (int e = 0; e < kEach; ++e) my_scales[e] = load_scales(my_blk[e]);
#pragma unroll
            for (int e = 0; e < kEach; ++e) store_meta(tid + kThreads * e, my_blk[e], my_scales[e]);
            __syncthreads();
            my_steps = steps_of(seg);
            first_steps(my_steps);
        }
        uint32_t slot = 0, free_slot = (kRing - 1) * S::kStage;  // ring bytes of the step in hand, and of the next to issue
        for (int k = 0; k < my_steps; ++k) {
            if (k + kRing - 1 < my_steps) issue((warp + kWarps * (k + kRing - 1)) * kStepGroups, free_slot);
            else cp_async_commit();
            free_slot = slot;
            cp_async_wait<kRing - 1>();
            __syncwarp();
            const unsigned char *blk0 = &sm.ring[warp][0][0] + slot;
            const int g0 = (warp + kWarps * k) * kStepGroups;
            float4 meta[kSub];
#pragma unroll
            for (int v = 0; v < kSub; ++v) meta[v] = sm.meta[g0 + kSubGroups * v + i4];

            // ---- scores of 16 tokens at a time: two tiles of 8 ------------------------------
            float2 x[HS][kSub][2];
            {
                // a chain per tile (9-16 heads: and part of q)
                float c[kSub][2][kChains][4];
                const unsigned char *kg = blk0 + (hl >> 1) * S::kBlk;
                uint32_t tiles[kSub][2];
#pragma unroll
                for (int v = 0; v < kSub; ++v) {
                    const unsigned char *at = kg + kSubGroups * v * S::kBlk + 4 * D + i4 * (D / 16);
                    if constexpr (D == 128) {
                        const uint2 two = *reinterpret_cast<const uint2 *>(at);
                        tiles[v][0] = two.x, tiles[v][1] = two.y;
                    } else {
                        tiles[v][0] = *reinterpret_cast<const uint32_t *>(at), tiles[v][1] = 0;
                    }
                }
#pragma unroll
                for (int j = 0; j < kHalves; ++j) {
                    uint4 q[kSub];
#pragma unroll
                    for (int v = 0; v < kSub; ++v)
                        q[v] = *reinterpret_cast<const uint4 *>(kg + kSubGroups * v * S::kBlk + (hl & 1) * 64 + i4 * 16 + j * 128);
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        uint32_t r[kSub][2][4];
#pragma unroll
                        for (int v = 0; v < kSub; ++v) {
                            const TileScale<F> ts(two_e4m3(tiles[v][j] >> (16 * w)));
                            decode_word<F>(w == 0 ? q[v].x : q[v].y, ts, int4_base, r[v][0]);
                            decode_word<F>(w == 0 ? q[v].z : q[v].w, ts, int4_base, r[v][1]);
                        }
#pragma unroll
                        for (int d = 0; d < 2; ++d)
#pragma unroll
                            for (int s = 0; s < HS; ++s) {  // (9-16 heads: q's hi, then its lo part)
                                const uint4 y = sm.qa[4 * j + 2 * w + d][s][lane];
                                const uint32_t qo[4] = {y.x, y.y, y.z, y.w};
                                const bool first = j == 0 && w == 0 && d == 0;
#pragma unroll
                                for (int v = 0; v < kSub; ++v)
#pragma unroll
                                    for (int t = 0; t < 2; ++t) {
                                        float (&ch)[4] = c[v][t][s];
                                        if (first) mma16816_first(ch, qo, r[v][t][2 * d], r[v][t][2 * d + 1]);
                                        else mma16816(ch, qo, r[v][t][2 * d], r[v][t][2 * d + 1]);
                                    }
                            }
                    }
                }
                // rows hl and hl+8 are the hi and lo parts of a head, or two heads
#pragma unroll
                for (int v = 0; v < kSub; ++v)
#pragma unroll
                    for (int s = 0; s < HS; ++s) {
                        const float f = hscale[s] * meta[v].x;
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            float2 y;
                            if constexpr (HS == 1) {
                                y = add2(make_float2(c[v][t][0][0], c[v][t][0][1]), make_float2(c[v][t][0][2], c[v][t][0][3]));
                            } else {
                                y = make_float2(c[v][t][0][2 * s], c[v][t][0][2 * s + 1]);
#pragma unroll
                                for (int n = 1; n < kChains; ++n) y = add2(y, make_float2(c[v][t][n][2 * s], c[v][t][n][2 * s + 1]));
                            }
                            x[s][v][t] = fma2s(y, f, meta[v].w);  // meta.w: -inf where there is no group
                        }
                    }
            }

            // ---- softmax of this lane's heads over the step, relative to mref ------------------
            // The reference follows the largest score only when that passes it by more than
            // 2^kLag, so that the accumulators are rescaled a few times in a row and not at almost
            // every step, and no lane needs to know the others' scores until one passes.
            uint32_t ph[HS][kSub][2], pl[HS][kSub][2];
            float xl[HS][kSub], gsum[HS][kSub], winv[HS];
            bool passed = false;
#pragma unroll
            for (int s = 0; s < HS; ++s)
#pragma unroll
                for (int v = 0; v < kSub; ++v) {
                    xl[s][v] = fmaxf(fmaxf(x[s][v][0].x, x[s][v][0].y), fmaxf(x[s][v][1].x, x[s][v][1].y));
                    passed = passed || xl[s][v] > m_pass[s];
                }
            if (__any_sync(0xffffffffu, passed)) {
#pragma unroll
                for (int s = 0; s < HS; ++s) {
                    float mc = xl[s][0];
#pragma unroll
                    for (int v = 1; v < kSub; ++v) mc = fmaxf(mc, xl[s][v]);
                    mc = fmaxf(mc, __shfl_xor_sync(0xffffffffu, mc, 1));
                    mc = fmaxf(mc, __shfl_xor_sync(0xffffffffu, mc, 2));
                    if (!(mc > m_pass[s])) mc = m_run[s];
                    const float alpha = mc == -INFINITY ? 1.0f : ex2(m_run[s] - mc);
                    m_run[s] = mc;
                    mref[s] = mc == -INFINITY ? 0.0f : mc;
                    m_pass[s] = mc + float(kLag);
                    l_run[s] *= alpha;
#pragma unroll
                    for (int j = 0; j < kVC; ++j)
#pragma unroll
                        for (int u = 0; u < 4; ++u) acc[s][j][u] = mul2(acc[s][j][u], alpha);
                }
            }
#pragma unroll
            for (int s = 0; s < HS; ++s) {
                // the largest log2 of a weight plus exponent of a V scale
                float zm = (xl[s][0] - mref[s]) + meta[0].z, wscale;
#pragma unroll
                for (int v = 1; v < kSub; ++v) zm = fmaxf(zm, (xl[s][v] - mref[s]) + meta[v].z);
                zm = fmaxf(zm, __shfl_xor_sync(0xffffffffu, zm, 1));
                zm = fmaxf(zm, __shfl_xor_sync(0xffffffffu, zm, 2));
                scale_of_weights<kLog2Units<F>>(zm, wscale, winv[s]);
#pragma unroll
                for (int v = 0; v < kSub; ++v) {
                    float2 p[2];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        p[t] = add2(x[s][v][t], make_float2(-mref[s], -mref[s]));
                        p[t] = make_float2(ex2(p[t].x), ex2(p[t].y));
                        split2(mul2(mul2(p[t], meta[v].y), wscale), ph[s][v][t], pl[s][v][t]);
                    }
                    const float2 g2 = add2(p[0], p[1]);
                    const float gs = g2.x + g2.y;
                    l_run[s] += gs;
                    gsum[s][v] = gs;
                }
            }
            if (a.mass != nullptr) {
#pragma unroll
                for (int s = 0; s < HS; ++s) {
#pragma unroll
                    for (int v = 0; v < kSub; ++v) {
                        const int h = hl + 8 * s, g = seg + g0 + kSubGroups * v;
                        if (h >= gq || g >= run_end) continue;
                        const int64_t hb = int64_t(b) * a.q_heads + h0 + h;
                        if (meta[v].w == 0.0f) a.mass[hb * a.mass_stride + g + i4] = gsum[s][v];
                        // (m_run itself: while it is -inf the masses are 0, and 2^(-inf - M) is 0 for every
                        // M, where 2^(0 - M) is infinite for M below -128 and would make the share NaN)
                        if (i4 == 0) a.mref[hb * (a.mass_stride / 4) + g / 4] = m_run[s];
                    }
                }
            }

            // ---- weighted values -------------------------------------------------------------
            uint32_t pa[kSub][4], pb[kSub][4];
#pragma unroll
            for (int v = 0; v < kSub; ++v)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    pa[v][2 * t] = ph[0][v][t];
                    pa[v][2 * t + 1] = HS == 1 ? pl[0][v][t] : ph[HS - 1][v][t];
                    pb[v][2 * t] = pl[0][v][t];  // (HS == 2)
                    pb[v][2 * t + 1] = pl[HS - 1][v][t];
                }
            const unsigned char *vp = blk0 + i4 * S::kBlk + 2 * D + hl * 16;
            const unsigned char *tp = blk0 + i4 * S::kBlk + 4 * D + D / 4 + hl * (D / 32);
            uint32_t tiles[kSub];
#pragma unroll
            for (int v = 0; v < kSub; ++v) {
                const unsigned char *at = tp + v * kSubGroups * S::kBlk;
                tiles[v] = D == 128 ? *reinterpret_cast<const uint32_t *>(at) : *reinterpret_cast<const uint16_t *>(at);
            }
#pragma unroll
            for (int m = 0; m < kHalves; ++m) {
                uint4 q[kSub];
                uint32_t two[kSub];
#pragma unroll
                for (int v = 0; v < kSub; ++v) {
                    q[v] = *reinterpret_cast<const uint4 *>(vp + v * kSubGroups * S::kBlk + m * 128);
                    two[v] = two_e4m3(tiles[v] >> (16 * m));
                }
                // kWords words at a time: word w has dims 64m + 32(w/2) + 4hl + 2(w%2) and + 1 of the lane's groups.
                // All products with one of the weights' operands come one after the other (up to 8 heads,
                // with the four words of a half at once: 8 histories of 262,144 tokens 140.8 -> 138.9 us)
                constexpr int kWords = HS == 1 ? 4 : 1;
#pragma unroll
                for (int w0 = 0; w0 < 4; w0 += kWords) {
                    float c[2 * kWords][4];
                    uint32_t r[kSub][kWords][4];
#pragma unroll
                    for (int v = 0; v < kSub; ++v) {
                        const uint32_t word[4] = {q[v].x, q[v].y, q[v].z, q[v].w};
#pragma unroll
                        for (int w = 0; w < kWords; ++w)
                            decode_word<F>(word[w0 + w], TileScale<F>(__byte_perm(two[v], 0, (w0 + w) / 2 == 0 ? 0x1010 : 0x3232)), int4_base, r[v][w]);
#pragma unroll
                        for (int u = 0; u < 2 * kWords; ++u) {
                            if (v == 0) mma16816_first(c[u], pa[0], r[0][u / 2][2 * (u % 2)], r[0][u / 2][2 * (u % 2) + 1]);
                            else mma16816(c[u], pa[v], r[v][u / 2][2 * (u % 2)], r[v][u / 2][2 * (u % 2) + 1]);
                        }
                    }
#pragma unroll
                    for (int u = 0; u < 2 * kWords; ++u) {
                        const int at = 2 * w0 + u, j = 2 * m + at / 4;  // dims 32j + 4hl + at%4
                        if constexpr (HS == 1) {
                            acc[0][j][at % 4] = fma2(add2(make_float2(c[u][0], c[u][1]), make_float2(c[u][2], c[u][3])), winv[0], acc[0][j][at % 4]);
                        } else {
#pragma unroll
                            for (int v = 0; v < kSub; ++v) mma16816(c[u], pb[v], r[v][u / 2][2 * (u % 2)], r[v][u / 2][2 * (u % 2) + 1]);
                            acc[0][j][at % 4] = fma2(make_float2(c[u][0], c[u][1]), winv[0], acc[0][j][at % 4]);
                            acc[HS - 1][j][at % 4] = fma2(make_float2(c[u][2], c[u][3]), winv[HS - 1], acc[HS - 1][j][at % 4]);
                        }
                    }
                }
            }
            __syncwarp();  // the slot is refilled by a later step
            slot = slot == (kRing - 1) * S::kStage ? 0 : slot + S::kStage;
        }
        cp_async_wait<0>();
    }
    // ---- the run's state: the warps' accumulators brought to one maximum and added in warp order
#pragma unroll
    for (int s = 0; s < HS; ++s) {
        float l = l_run[s];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (i4 == 0) {
            sm.wm[warp][hl + 8 * s] = m_run[s];
            sm.wl[warp][hl + 8 * s] = l;
        }
    }
    __syncthreads();  // (and every warp is done with the ring)
    float *red = reinterpret_cast<float *>(sm.ring);  // [kWarps][kNH][D]
    const int64_t pbase = (int64_t(b) * a.q_heads + h0) * a.nparts + part;  // of the first head
#pragma unroll
    for (int s = 0; s < HS; ++s) {
        const int h = hl + 8 * s;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.wm[w][h]);
        const float Ms = M == -INFINITY ? 0.0f : M;
        const float wt = ex2(m_run[s] - Ms);
        if (warp == 0 && i4 == 0 && h < gq) {
            float L = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) L = fmaf(sm.wl[w][h], ex2(sm.wm[w][h] - Ms), L);
            a.part_m[pbase + int64_t(h) * a.nparts] = M;
            a.part_l[pbase + int64_t(h) * a.nparts] = L;
        }
#pragma unroll
        for (int j = 0; j < kVC; ++j) {
#pragma unroll
            for (int u = 0; u < 4; ++u) acc[s][j][u] = mul2(acc[s][j][u], wt);
            float4 *dst = reinterpret_cast<float4 *>(red + (warp * kNH + h) * D + 32 * j + 8 * i4);
            dst[0] = make_float4(acc[s][j][0].x, acc[s][j][1].x, acc[s][j][2].x, acc[s][j][3].x);
            dst[1] = make_float4(acc[s][j][0].y, acc[s][j][1].y, acc[s][j][2].y, acc[s][j][3].y);
        }
    }
    __syncthreads();
    constexpr int F4 = D / 4;
    for (int e = tid; e < gq * F4; e += kThreads) {
        const int h = e / F4, c = e % F4;
        float4 o = *reinterpret_cast<const float4 *>(red + h * D + 4 * c);
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            const float4 p = *reinterpret_cast<const float4 *>(red + (w * kNH + h) * D + 4 * c);
            o.x += p.x;
            o.y += p.y;
            o.z += p.z;
            o.w += p.w;
        }
        reinterpret_cast<float4 *>(a.part_acc + (pbase + int64_t(h) * a.nparts) * D)[c] = o;
    }
}

template <int D, int HS, int F>
cudaError_t launch_t(const AttendCodedArgs &a, int runs, cudaStream_t s)
{
    using S = Sm<D, HS, F>;
    static_assert(sizeof(S) <= 227 * 1024, "shared memory per CTA");
    static_assert(ctas_per_sm<D, HS>() * (sizeof(S) + 1024) <= 228 * 1024, "the CTAs per SM that the kernels are built for");
    static_assert(kSegGroups % kThreads == 0, "groups that a thread resolves");
    static_assert(kWarps * 8 * HS * D * 4 <= int(sizeof(S::ring)), "the reduction area fits the ring");
    const size_t smem = sizeof(S);
    static bool attr_done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_done[dev]) {
        e = cudaFuncSetAttribute(attend_coded4_kernel<D, HS, F>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return e;
        attr_done[dev] = true;
    }
    return launch_kernel(attend_coded4_kernel<D, HS, F>, dim3(unsigned(runs + (a.sharing != nullptr ? 2 : 1)) * unsigned(a.kv_heads), 1, unsigned(a.batch)),
                         dim3(kThreads), smem, s, true, a);
}

template <int F>
cudaError_t launch_format(const AttendCodedArgs &a, int runs, cudaStream_t s)
{
    const bool one = a.q_heads / a.kv_heads <= 8;
    if (a.head_dim == 128) return one ? launch_t<128, 1, F>(a, runs, s) : launch_t<128, 2, F>(a, runs, s);
    return one ? launch_t<64, 1, F>(a, runs, s) : launch_t<64, 2, F>(a, runs, s);
}

}  // namespace

cudaError_t launch_attend_coded4(const AttendCodedArgs &a, int runs, cudaStream_t s)
{
    return a.format == QSA_CODE_INT4 ? launch_format<QSA_CODE_INT4>(a, runs, s) : launch_format<QSA_CODE_E2M1>(a, runs, s);
}

}  // namespace qsa
