// attend_coded.cu -- attention of one query per batch entry over K/V rows held
// in 8-bit codes with a scale per (group, KV head) (include/qsa_cache.h:
// qsa_attend_coded), with the attention that each group received.
//
// Mathematics.  x_t = scale * sK_g * (q . kcode_t), p_t = e^(x_t - m), out =
// sum_t p_t sV_g vcode_t / sum_t p_t, as an online softmax: a running maximum
// m, denominator and accumulator per warp, merged over the warps of a run and
// over the runs of a row in a fixed order.
//
// An 8-bit code is exact in a 16-bit float, so both products run on the tensor
// cores with operands of 22 bits: q and the weights w_t = p_t sV_g enter as
// hi + lo, two 16-bit floats of 11 bits each, under a power of two per head (q) or
// per head and step (w) that brings the largest to 2^12 or more, so that what falls
// among the 16-bit subnormals is below 2^-37 of it.  (A power of two per step alone,
// from its largest sV, lost the groups that a head attends to beside larger ones:
// 1 % of the output at sV 2^-24 of a neighbour's, all of it at 2^-32.)  The
// matrix instruction m16n8k16 has 16 rows; with at most 8 query heads per KV
// head, rows 0-7 hold the hi parts and rows 8-15 the lo parts of the same heads,
// so one instruction does both and its two result rows h and h+8, which the same
// lane holds, add up to the product.  (9 to 16 heads: rows are heads, and the lo
// parts have sums of their own.)  The tensor core's own sums may
// truncate, so a chain covers 16 tokens, or d dims, and starts from zero; its
// result goes into the binary32 running sums by additions that round to nearest.
//
// Layout.  A warp step is 4 groups (16 tokens).  For the first product tile t
// holds tokens 2t, 2t+1 of the 4 groups (column n: group n/2, token 2t + n%2),
// so a lane (head = lane/4, i = lane%4) ends with the scores of group i's four
// tokens for its head: the group's share of attention is a sum within the lane,
// and the four weights are the operand of the second product as they stand.
// Its other operand, the codes of one dim for the four tokens of a group, is
// one word of the V layout.  A block of codes sits in shared memory with 32
// bytes behind it: the 16-byte reads of both products are free of conflicts.
//
// Data movement.  A CTA of four warps takes one run of a row; each warp streams
// its own steps through a ring of two (16-byte asynchronous copies, a step ahead
// of its arithmetic), so there is no block barrier in the loop.  Four CTAs per SM
// (128 registers) cover one another's starts -- the row, its blocks, their scales
// and the query are three dependent loads -- and ends.
//
// Bound: 8*d + 8 bytes per (group, KV head), read once.  8 histories of 262,144
// tokens (16 / 2 heads x 128, e4m3, 1.08 GB): 179 us of this kernel, 6.1 TB/s, the
// tensor pipe 25-30 % and the issue slots about half busy; with the blocks in
// order instead of permuted 7 % less, the rest of the distance to the copy rate
// (6.77 TB/s) being starts and ends.  Rows of a few thousand tokens and selected
// rows (512 groups: 5.4 us for 8 queries) are bound by a CTA's start and end.
// Tried and not kept: a ring of three (189 us), copies by the bulk engine (its
// operands are uniform, so four lanes' copies are issued one after the other:
// 60 more instructions a step, 188 us), resident CTAs that take several runs with
// the next run's addresses loaded ahead (199-207 us: a fixed share of the runs
// waits for the slowest SM), two runs of selected rows per CTA, five CTAs per SM
// with q read from shared memory at each step (191 us), runs merged by the last CTA of
// a row (rows of 512 groups 7.3 -> 10.5 us a call) or by the only one (37 tokens 6.4
// -> 8.3 us on the device), the last eighth of a row in short runs (187 us).
#include <cuda_fp16.h>

#include "cache_internal.cuh"

namespace qsa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStepGroups = 4;                  // groups per warp step
constexpr int kRing = 2;                        // a warp's steps in shared memory: one in use, one on its way
constexpr int kSegGroups = 128;                 // groups resolved at a time
constexpr int kBlkPad = 32;                     // bytes behind a block in shared memory

template <int D, int HS>
struct Sm {
    static constexpr int kBlk = 8 * D + kBlkPad;
    static constexpr int kStage = kStepGroups * kBlk;
    alignas(128) unsigned char ring[kWarps][kRing][kStage];  // also the end-of-run reduction area
    alignas(16) float4 meta[kSegGroups];                     // K scale, V scale and its exponent, 0 (-inf: no such group)
    alignas(16) uint4 qa[D / 16][HS][32];                    // each lane's operands of q (9-16 heads: hi, lo)
    float qs[8 * HS];                                        // 1/f of each head's q
    alignas(16) int blk[kSegGroups];                         // physical block; -1: none, -2: zero rows
    float wm[kWarps][8 * HS], wl[kWarps][8 * HS];
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// c += a * b, or (first) c = a * b.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// Two binary32 operations in one instruction, each rounded to nearest.
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 r;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2s(float2 a, float b, float c)  // a * b + c
{
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tmov.b64 z, {%5, %5};\n\tfma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float b)
{
    float2 r;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float b, float2 c)
{
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tmov.b64 z, {%5, %6};\n\tfma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b), "f"(c.x), "f"(c.y));
    return r;
}

// Four codes as two pairs of 16-bit floats (exact).
template <bool kInt8>
__device__ __forceinline__ void decode4(uint32_t w, uint32_t &b0, uint32_t &b1)
{
    if constexpr (kInt8) {
        // code + 128 under the exponent of 1024 is 1024 + 128 + code
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
        const uint32_t k = 0x64806480u;  // 1152, 1152
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(b0) : "r"(lo), "r"(k));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(b1) : "r"(hi), "r"(k));
    } else {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(b0), "=r"(b1)
            : "r"(w));
    }
}

// x and y as hi and lo pairs of 16-bit floats: hi + lo is x to 22 bits.
__device__ __forceinline__ void split2(float2 v, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __floats2half2_rn(v.x, v.y);
    const float2 f = __half22float2(h);
    const float2 r = add2(v, make_float2(-f.x, -f.y));
    const __half2 l = __floats2half2_rn(r.x, r.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}

// The power of two that brings the largest magnitude of a head's q (its bits) to
// [2^13, 2^14), and its inverse.  The exponent is kept to -110..128, so that both are
// normal floats.
__device__ __forceinline__ void scale_of_q(uint32_t top, float &f, float &inv)
{
    const int e = max(int(top >> 23) - 127, -110);
    f = __uint_as_float(uint32_t(13 - e + 127) << 23);
    inv = __uint_as_float(uint32_t(e - 13 + 127) << 23);
}

// The same for the weights of a head in a step, to [2^12, 2^15).  z: the largest sum of
// a softmax weight's log2 and a V scale's exponent, so that the largest weight is
// 2^z to 2^(z+1); at most 16 + 121, and NaN where every weight is (any power will do).
// The sum with 1.5 * 2^23 rounds z to an integer and holds it in its low bits.
__device__ __forceinline__ void scale_of_weights(float z, float &f, float &inv)
{
    const uint32_t e = __float_as_uint(__fadd_rn(fmaxf(z, -110.0f), 12582912.0f));
    const uint32_t bits = (uint32_t(13 + 127) << 23) - (e << 23);
    f = __uint_as_float(bits);
    inv = __uint_as_float((uint32_t(2 * 127) << 23) - bits);
}

constexpr int kLag = 8;     // log2 of the largest softmax weight (16 where the scores' own rounding is that coarse)

// CTAs per SM that the registers and the ring leave room for.
template <int D, int HS>
constexpr int ctas_per_sm() { return HS == 2 ? 3 : D == 128 ? 4 : 6; }

// Whether query b's row may add weights, and to whose accumulators; by a whole CTA.
__device__ __forceinline__ void find_sharing(const AttendCodedArgs &a, int b, const Row &row)
{
    const int tid = threadIdx.x;
    int bad = row.ok ? 0 : 1;
    if (a.ids != nullptr) {  // its groups are well formed and ascend
        const int32_t *ids = a.ids + int64_t(b) * a.row_cap;
#pragma unroll 4
        for (int g = tid; g < row.groups; g += kThreads) {
            int id[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) id[u] = __ldcg(ids + kGroup * g + u);
            const int last = __ldcg(ids + max(kGroup * g - 4, 0));
            bad |= int(id[0] < 0) | int(id[0] % kGroup != 0) | int(id[0] > row.T - kGroup) | int(id[1] != id[0] + 1) |
                   int(id[2] != id[0] + 2) | int(id[3] != id[0] + 3) | int(g > 0 && last >= id[0]);
        }
        if (tid < row.tail) {
            const int id = __ldcg(ids + kGroup * row.groups + tid);
            bad |= int(id < 0) | int(id >= row.T) | int(id / kGroup != row.T / kGroup);
        }
    }
    // its own accumulators, or those of several queries
    const int64_t off = __ldg(a.weight_offset + b);
    int earlier = 0, later = 0;
#pragma unroll 4
    for (int o = tid; o < a.batch; o += kThreads) {
        const int same = int(__ldg(a.weight_offset + o) == off);
        earlier |= same & int(o < b);
        later |= same & int(o > b);
    }
    bad = __syncthreads_or(bad);
    earlier = __syncthreads_or(earlier);
    later = __syncthreads_or(later);
    if (tid == 0) {
        a.sharing[b] = (bad ? kBad : 0u) | (earlier ? kLaterSharer : later ? kFirstSharer : 0u);
        if (bad && row.ok) set_error(a.err, QSA_DEVERR_ROW_RANGE);
    }
}

// The raw tail of query b for the heads of one KV head, at most 3 tokens in
// binary32: one more run, a warp per head.
template <int D>
__device__ __forceinline__ void attend_tail(const AttendCodedArgs &a, int b, int kvh, const Row &row, int run)
{
    constexpr int kPer = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gq = a.q_heads / a.kv_heads;
    int slot = -1;  // lane u < tail: of token u
    if (lane < row.tail) {
        const int64_t at = int64_t(b) * a.row_cap + kGroup * int64_t(row.groups) + lane;
        const int id = a.ids == nullptr ? kGroup * row.groups + lane : __ldcg(a.ids + at);
        if (kvh == 0 && warp == 0 && a.ids_out != nullptr) a.ids_out[at] = id;
        if (id < 0 || id >= row.T) {
            set_error(a.err, QSA_DEVERR_ROW_RANGE);
        } else {
            slot = __ldg(a.slot_map + __ldg(a.slot_offset + b) + id);
            if (slot < 0 || slot >= a.num_slots) {
                set_error(a.err, QSA_DEVERR_SLOT_RANGE);
                slot = -1;
            }
        }
    }
    float k[3][kPer], v[3][kPer];
#pragma unroll
    for (int u = 0; u < 3; ++u) {
        const int sl = __shfl_sync(0xffffffffu, slot, u);
        const int64_t at = (int64_t(sl) * a.kv_heads + kvh) * D + lane;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            k[u][j] = sl >= 0 ? __ldg(a.k_cache + at + 32 * j) : 0.0f;
            v[u][j] = sl >= 0 ? __ldg(a.v_cache + at + 32 * j) : 0.0f;
        }
    }
    for (int h = warp; h < gq; h += kWarps) {
        const int64_t hb = int64_t(b) * a.q_heads + kvh * gq + h;
        float q[kPer], x[3], p[3], m = -INFINITY, l = 0.0f;
#pragma unroll
        for (int j = 0; j < kPer; ++j) q[j] = __ldg(a.q + hb * D + lane + 32 * j);
#pragma unroll
        for (int u = 0; u < 3; ++u) {
            float dot = 0.0f;
#pragma unroll
            for (int j = 0; j < kPer; ++j) dot = fmaf(q[j], k[u][j], dot);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
            x[u] = u < row.tail ? dot * (a.scale * kLog2e) : -INFINITY;
            m = fmaxf(m, x[u]);
        }
        const float ms = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int u = 0; u < 3; ++u) {
            p[u] = u < row.tail ? ex2(x[u] - ms) : 0.0f;
            l += p[u];
        }
        float *acc = a.part_acc + (hb * a.nparts + run) * D;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            float o = 0.0f;
#pragma unroll
            for (int u = 0; u < 3; ++u)
                if (u < row.tail) o = fmaf(p[u], v[u][j], o);
            acc[lane + 32 * j] = o;
        }
        if (lane == 0) {
            a.part_m[hb * a.nparts + run] = m;
            a.part_l[hb * a.nparts + run] = l;
        }
    }
}

template <int D, int HS, bool kInt8>
__global__ void __launch_bounds__(kThreads, (ctas_per_sm<D, HS>())) attend_coded_kernel(const AttendCodedArgs a)
{
    extern __shared__ __align__(128) unsigned char smem_raw[];
    using S = Sm<D, HS>;
    S &sm = *reinterpret_cast<S *>(smem_raw);
    constexpr int kNH = 8 * HS;
    constexpr int kHalves = D / 64;       // 64-dim halves of K
    constexpr int kVC = D / 32;           // 16-byte V reads per lane and group
    constexpr int kChains = HS == 1 ? 1 : 2 * kHalves;  // independent accumulations of a score tile

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int hl = lane >> 2, i4 = lane & 3;
    const int gq = a.q_heads / a.kv_heads;
    const bool whole = a.ids == nullptr;

    wait_for_predecessor();
    // the first CTAs of each (query, KV head): the raw tail, and what belongs to the query as a whole
    const int extra = a.sharing != nullptr ? 2 : 1;
    const int part = int(blockIdx.x) - extra, kvh = blockIdx.y, b = blockIdx.z;
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
        const int ctas = (int(gridDim.x) - extra) * a.kv_heads, n = (a.map_stride / 4 + ctas - 1) / ctas;
        const int g0 = (part * a.kv_heads + kvh) * n;
        float4 *map = reinterpret_cast<float4 *>(a.share_map + int64_t(b) * a.map_stride);
        for (int g = g0 + tid; g < min(g0 + n, a.map_stride / 4); g += kThreads) map[g] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int per_run = coded_run_groups(row.groups, whole, gq);
    const int run_begin = part * per_run, run_end = min(row.groups, run_begin + per_run);
    if (run_begin >= run_end) return;

    // A run is taken in segments of up to kSegGroups groups, thread t resolving group
    // seg + t: its block first, so that copies can start, ...
    auto load_block = [&](int seg) {
        int g = seg + tid;
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
    auto store_meta = [&](int blk, float2 sc) {
        const uint32_t bits = __float_as_uint(sc.y) & 0x7fffffffu;
        const float e = bits == 0 ? -INFINITY : float(int(bits >> 23) - 127);
        sm.meta[tid] = make_float4(sc.x, sc.y, e, blk != -1 ? 0.0f : -INFINITY);
    };
    const unsigned char *codes = a.codes + int64_t(kvh) * (8 * D) + lane * 16;  // this lane's first piece of block 0
    const int64_t blk_bytes = int64_t(a.kv_heads) * (8 * D);
    const uint32_t ring = smem_u32(sm.ring[warp]) + lane * 16;
    auto issue = [&](int g0, uint32_t slot) {  // the step at group g0 of the segment, into ring bytes slot
        const int4 blks = *reinterpret_cast<const int4 *>(sm.blk + g0);
        const int blk[4] = {blks.x, blks.y, blks.z, blks.w};
        if (min(min(blk[0], blk[1]), min(blk[2], blk[3])) >= 0) {
            if constexpr (D == 128) {  // a block is two pieces per lane
#pragma unroll
                for (int u = 0; u < kStepGroups; ++u) {
                    const unsigned char *src = codes + blk[u] * blk_bytes;
                    cp_async16(ring + slot + u * S::kBlk, src);
                    cp_async16(ring + slot + u * S::kBlk + 512, src + 512);
                }
            } else {
#pragma unroll
                for (int u = 0; u < kStepGroups; ++u) cp_async16(ring + slot + u * S::kBlk, codes + blk[u] * blk_bytes);
            }
        } else {  // some groups are not there, or not to be read: zeros
            for (int u = 0; u < kStepGroups; ++u) {
                const int bu = sm.blk[g0 + u];
                for (int c = 0; c < 8 * D; c += 512) {
                    if (bu >= 0) cp_async16(ring + slot + u * S::kBlk + c, codes + bu * blk_bytes + c);
                    else *reinterpret_cast<uint4 *>(&sm.ring[warp][0][0] + slot + u * S::kBlk + c + lane * 16) = make_uint4(0, 0, 0, 0);
                }
            }
        }
        cp_async_commit();
    };
    // this warp's steps of a segment: groups 4 * (warp + kWarps * k)
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

    int my_blk = load_block(run_begin);
    sm.blk[tid] = my_blk;
    __syncthreads();
    int my_steps = steps_of(run_begin);
    first_steps(my_steps);
    const float2 my_scales = load_scales(my_blk);

    // ---- the queries: 16 threads a head, each 8 dims at a time, to the matrix operands -----
    // of the lane that holds the dims: words of dims 4u..4u+3 of 64j + 16*i4, hi and lo,
    // with the head's power of two taken out
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
        split2(make_float2(x.x * f, x.y * f), hi[0], lo[0]);
        split2(make_float2(x.z * f, x.w * f), hi[1], lo[1]);
        split2(make_float2(y.x * f, y.y * f), hi[2], lo[2]);
        split2(make_float2(y.z * f, y.w * f), hi[3], lo[3]);
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
    store_meta(my_blk, my_scales);
    __syncthreads();
    uint32_t qa[HS == 1 ? kHalves : 1][4][4];  // (up to 8 heads: in registers)
    if constexpr (HS == 1) {
#pragma unroll
        for (int j = 0; j < kHalves; ++j)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint4 v = sm.qa[4 * j + u][0][lane];
                qa[j][u][0] = v.x, qa[j][u][1] = v.y, qa[j][u][2] = v.z, qa[j][u][3] = v.w;
            }
    }
    float hscale[HS];
#pragma unroll
    for (int s = 0; s < HS; ++s) hscale[s] = a.scale * kLog2e * sm.qs[hl + 8 * s];

    // the accumulator: dims 32*j + 8*i4 + u (x) and + 4 (y) of head hl + 8*s
    float2 acc[HS][kVC][4];
    float m_run[HS], l_run[HS];
#pragma unroll
    for (int s = 0; s < HS; ++s) {
        m_run[s] = -INFINITY;
        l_run[s] = 0.0f;
#pragma unroll
        for (int j = 0; j < kVC; ++j)
#pragma unroll
            for (int u = 0; u < 4; ++u) acc[s][j][u] = make_float2(0.0f, 0.0f);
    }

    for (int seg = run_begin; seg < run_end; seg += kSegGroups) {
        if (seg != run_begin) {  // every warp is done with the last segment's blocks
            __syncthreads();
            my_blk = load_block(seg);
            sm.blk[tid] = my_blk;
            store_meta(my_blk, load_scales(my_blk));
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
            const float4 meta = sm.meta[g0 + i4];

            // ---- scores of the step's 16 tokens: two tiles of 8 ---------------------------
            float2 x[HS][2];
            {
                float c[2][kChains][4];  // up to 8 heads: a chain per tile; else one per tile, 64 dims and part of q (51.6 us against 52.9)
                const unsigned char *kp = blk0 + (hl >> 1) * S::kBlk + (hl & 1) * 64 + i4 * 16;
#pragma unroll
                for (int j = 0; j < kHalves; ++j) {
                    uint32_t w[2][4];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(kp + j * 256 + t * 128);
                        w[t][0] = v.x;
                        w[t][1] = v.y;
                        w[t][2] = v.z;
                        w[t][3] = v.w;
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        uint32_t qh[4], ql[4];
                        if constexpr (HS == 2) {
                            const uint4 v = sm.qa[4 * j + u][0][lane], z = sm.qa[4 * j + u][1][lane];
                            qh[0] = v.x, qh[1] = v.y, qh[2] = v.z, qh[3] = v.w;
                            ql[0] = z.x, ql[1] = z.y, ql[2] = z.z, ql[3] = z.w;
                        }
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            uint32_t b0, b1;
                            decode4<kInt8>(w[t][u], b0, b1);
                            if constexpr (HS == 1) {
                                if (j == 0 && u == 0) mma16816_first(c[t][0], qa[j][u], b0, b1);
                                else mma16816(c[t][0], qa[j][u], b0, b1);
                            } else {
                                float (&ch)[4] = c[t][HS == 1 ? 0 : 2 * j], (&cl)[4] = c[t][HS == 1 ? 0 : 2 * j + 1];
                                if (u == 0) mma16816_first(ch, qh, b0, b1);
                                else mma16816(ch, qh, b0, b1);
                                if (u == 0) mma16816_first(cl, ql, b0, b1);
                                else mma16816(cl, ql, b0, b1);
                            }
                        }
                    }
                }
                // rows hl and hl+8 are the hi and lo parts of a head, or two heads
#pragma unroll
                for (int s = 0; s < HS; ++s) {
                    const float f = hscale[s] * meta.x;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        float2 v;
                        if constexpr (HS == 1) {
                            v = add2(make_float2(c[t][0][0], c[t][0][1]), make_float2(c[t][0][2], c[t][0][3]));
                        } else {
                            v = make_float2(c[t][0][2 * s], c[t][0][2 * s + 1]);
#pragma unroll
                            for (int n = 1; n < kChains; ++n) v = add2(v, make_float2(c[t][n][2 * s], c[t][n][2 * s + 1]));
                        }
                        x[s][t] = fma2s(v, f, meta.w);  // meta.w: -inf where there is no group
                    }
                }
            }

            // ---- softmax of this lane's heads over the step, relative to m_run ----------------
            // m_run follows the largest score only when that passes it by more than
            // 2^kLag, so that the accumulators are rescaled a few times in a row and
            // not at almost every step; weights stay below 2^kLag.
            uint32_t ph[HS][2], pl[HS][2];
            // zm: the largest log2 of a weight plus exponent of a V scale, as m_run stands
            float xl[HS], mc[HS], zm[HS], winv[HS];
            bool passed = false;
            auto reference = [&](int s) { return m_run[s] == -INFINITY ? 0.0f : m_run[s]; };
#pragma unroll
            for (int s = 0; s < HS; ++s) {
                xl[s] = fmaxf(fmaxf(x[s][0].x, x[s][0].y), fmaxf(x[s][1].x, x[s][1].y));
                mc[s] = fmaxf(xl[s], __shfl_xor_sync(0xffffffffu, xl[s], 1));
                zm[s] = (xl[s] - reference(s)) + meta.z;
                zm[s] = fmaxf(zm[s], __shfl_xor_sync(0xffffffffu, zm[s], 1));
                mc[s] = fmaxf(mc[s], __shfl_xor_sync(0xffffffffu, mc[s], 2));
                zm[s] = fmaxf(zm[s], __shfl_xor_sync(0xffffffffu, zm[s], 2));
                passed = passed || mc[s] > m_run[s] + float(kLag);
            }
            if (__any_sync(0xffffffffu, passed)) {
#pragma unroll
                for (int s = 0; s < HS; ++s) {
                    if (!(mc[s] > m_run[s] + float(kLag))) mc[s] = m_run[s];
                    const float alpha = mc[s] == -INFINITY ? 1.0f : ex2(m_run[s] - mc[s]);
                    m_run[s] = mc[s];
                    zm[s] = (xl[s] - reference(s)) + meta.z;
                    zm[s] = fmaxf(zm[s], __shfl_xor_sync(0xffffffffu, zm[s], 1));
                    zm[s] = fmaxf(zm[s], __shfl_xor_sync(0xffffffffu, zm[s], 2));
                    l_run[s] *= alpha;
#pragma unroll
                    for (int j = 0; j < kVC; ++j)
#pragma unroll
                        for (int u = 0; u < 4; ++u) acc[s][j][u] = mul2(acc[s][j][u], alpha);
                }
            }
#pragma unroll
            for (int s = 0; s < HS; ++s) {
                const float ms = reference(s);
                float f;
                scale_of_weights(zm[s], f, winv[s]);
                float2 p[2];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    p[t] = add2(x[s][t], make_float2(-ms, -ms));
                    p[t] = make_float2(ex2(p[t].x), ex2(p[t].y));
                }
                const float gs = (p[0].x + p[0].y) + (p[1].x + p[1].y);
                l_run[s] += gs;
                split2(mul2(mul2(p[0], meta.y), f), ph[s][0], pl[s][0]);
                split2(mul2(mul2(p[1], meta.y), f), ph[s][1], pl[s][1]);
                const int h = hl + 8 * s;
                if (a.mass != nullptr && h < gq) {
                    const int64_t hb = int64_t(b) * a.q_heads + h0 + h;
                    if (meta.w == 0.0f) a.mass[hb * a.mass_stride + seg + g0 + i4] = gs;
                    // (m_run itself: while it is -inf the masses are 0, and 2^(-inf - M) is 0 for every
                    // M, where 2^(0 - M) is infinite for M below -128 and would make the share NaN)
                    if (i4 == 0) a.mref[hb * (a.mass_stride / 4) + (seg + g0) / 4] = m_run[s];
                }
            }

            // ---- weighted values -------------------------------------------------------------
            const uint32_t pa[4] = {ph[0][0], HS == 1 ? pl[0][0] : ph[HS - 1][0], ph[0][1], HS == 1 ? pl[0][1] : ph[HS - 1][1]};
            const uint32_t pb[4] = {pl[0][0], pl[HS - 1][0], pl[0][1], pl[HS - 1][1]};  // (HS == 2)
            const unsigned char *vp = blk0 + i4 * S::kBlk + 4 * D + hl * 16;
#pragma unroll
            for (int j = 0; j < kVC; ++j) {
                const uint4 v = *reinterpret_cast<const uint4 *>(vp + j * 128);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint32_t b0, b1;
                    decode4<kInt8>(w[u], b0, b1);
                    float c[4];
                    mma16816_first(c, pa, b0, b1);
                    if constexpr (HS == 1) {
                        acc[0][j][u] = fma2(add2(make_float2(c[0], c[1]), make_float2(c[2], c[3])), winv[0], acc[0][j][u]);
                    } else {
                        mma16816(c, pb, b0, b1);
                        acc[0][j][u] = fma2(make_float2(c[0], c[1]), winv[0], acc[0][j][u]);
                        acc[HS - 1][j][u] = fma2(make_float2(c[2], c[3]), winv[HS - 1], acc[HS - 1][j][u]);
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

template <int D, int HS, bool kInt8>
cudaError_t launch_t(const AttendCodedArgs &a, int runs, cudaStream_t s)
{
    const size_t smem = sizeof(Sm<D, HS>);
    static bool attr_done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_done[dev]) {
        e = cudaFuncSetAttribute(attend_coded_kernel<D, HS, kInt8>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return e;
        attr_done[dev] = true;
    }
    return launch_kernel(attend_coded_kernel<D, HS, kInt8>, dim3(unsigned(runs + (a.sharing != nullptr ? 2 : 1)), unsigned(a.kv_heads), unsigned(a.batch)),
                         dim3(kThreads), smem, s, true, a);
}

static_assert(sizeof(Sm<128, 2>) <= 227 * 1024, "shared memory per CTA");
static_assert(4 * (sizeof(Sm<128, 1>) + 1024) <= 228 * 1024 && 3 * (sizeof(Sm<128, 2>) + 1024) <= 228 * 1024 &&
                  6 * (sizeof(Sm<64, 1>) + 1024) <= 228 * 1024, "the CTAs per SM that the kernels are built for");
static_assert(kThreads == kSegGroups, "a thread resolves a group");
static_assert(kWarps * 16 * 128 * 4 <= int(sizeof(Sm<128, 2>::ring)) && kWarps * 16 * 64 * 4 <= int(sizeof(Sm<64, 2>::ring)),
              "the reduction area fits the ring");

}  // namespace

bool attend_coded_shape_supported(int head_dim, int q_heads, int kv_heads)
{
    return (head_dim == 64 || head_dim == 128) && q_heads / kv_heads <= kMaxGqa && kv_heads <= 65535;
}

cudaError_t launch_attend_coded(const AttendCodedArgs &a, cudaStream_t s)
{
    if (a.batch == 0) return cudaSuccess;
    const bool whole = a.ids == nullptr;
    const int runs = coded_max_runs(whole ? a.max_visible / kGroup : (a.row_cap - (kGroup - 1)) / kGroup, whole,
                                    a.q_heads / a.kv_heads);
    const bool one = a.q_heads / a.kv_heads <= 8, i8 = a.format == QSA_CODE_INT8;
    cudaError_t e;
    if (a.head_dim == 128)
        e = one ? (i8 ? launch_t<128, 1, true>(a, runs, s) : launch_t<128, 1, false>(a, runs, s))
                : (i8 ? launch_t<128, 2, true>(a, runs, s) : launch_t<128, 2, false>(a, runs, s));
    else
        e = one ? (i8 ? launch_t<64, 1, true>(a, runs, s) : launch_t<64, 1, false>(a, runs, s))
                : (i8 ? launch_t<64, 2, true>(a, runs, s) : launch_t<64, 2, false>(a, runs, s));
    if (e != cudaSuccess) return e;
    return launch_merge_coded(a, s);
}

}  // namespace qsa
