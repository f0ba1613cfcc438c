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
// cores with operands that lose nothing: q and the weights w_t = p_t sV_g enter
// as hi + lo, two 16-bit floats of 11 bits each, scaled by a power of two so
// that the larger of them sits near 2^14 (both halves stay clear of the 16-bit
// subnormals).  The matrix instruction m16n8k16 has 16 rows; with at most 8
// query heads per KV head, rows 0-7 hold the hi parts and rows 8-15 the lo
// parts of the same heads, so one instruction does both and its two result rows
// h and h+8, which the same lane holds, add up to the product.  (9 to 16 heads:
// rows are heads, and the lo parts follow the hi parts into the same sum.)  Every instruction chain starts from zero and its result is added
// to the binary32 running sums by ordinary additions, which round to nearest.
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
// Bound by memory: 8*d + 8 bytes per (group, KV head), read once.
#include <cuda_fp16.h>

#include "cache_internal.cuh"

namespace qsa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStepGroups = 4;                  // groups per warp step
constexpr int kRing = 3;                        // steps in flight per warp
constexpr int kSegGroups = 128;                 // groups resolved at a time
constexpr int kBlkPad = 32;                     // bytes behind a block in shared memory
constexpr float kLog2e = 1.4426950408889634f;

template <int D, int HS>
struct Sm {
    static constexpr int kBlk = 8 * D + kBlkPad;
    static constexpr int kStage = kStepGroups * kBlk;
    alignas(128) unsigned char ring[kWarps][kRing][kStage];  // also the end-of-run reduction area
    alignas(16) float4 meta[kSegGroups];                     // K scale, V scale * f, 1/f, 1 if the group is there
    alignas(16) uint4 qa[HS == 2 ? D / 16 : 1][2][32];       // 9-16 heads: each lane's operands of q, hi and lo
    alignas(8) uint64_t full[kWarps][kRing];                 // a step's blocks have landed
    int blk[kSegGroups];                                     // physical block; -1: none, -2: zero rows
    float wm[kWarps][8 * HS], wl[kWarps][8 * HS], ww[kWarps][8 * HS];
    int traw[4];
};

// 2^x; results below the smallest normal float are 0.
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

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
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}

// Powers of two that bring a largest magnitude (its bits) to [2^kTop / 2, 2^kTop),
// and back.  The exponent is kept to -110..128, so that both are normal floats.
constexpr int kQTop = 14;   // of q
constexpr int kLag = 8;     // log2 of the largest softmax weight
constexpr int kVTop = 6;    // of the V scales of a step: times a weight, below 2^14
template <int kTop>
__device__ __forceinline__ void scale_to(uint32_t top, float &f, float &inv)
{
    const int e = max(int(top >> 23) - 127, -110);
    f = __uint_as_float(uint32_t(kTop - 1 - e + 127) << 23);
    inv = __uint_as_float(uint32_t(e - kTop + 1 + 127) << 23);
}

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

template <int D, int HS, bool kInt8>
__global__ void __launch_bounds__(kThreads, HS == 1 ? 4 : 2) attend_coded_kernel(const AttendCodedArgs a)
{
    extern __shared__ __align__(128) unsigned char smem_raw[];
    using S = Sm<D, HS>;
    S &sm = *reinterpret_cast<S *>(smem_raw);
    constexpr int kNH = 8 * HS;
    constexpr int kHalves = D / 64;       // 64-dim halves of K
    constexpr int kVC = D / 32;           // 16-byte V reads per lane and group

    const int part = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int hl = lane >> 2, i4 = lane & 3;
    const int gq = a.q_heads / a.kv_heads;
    const int h0 = kvh * gq;
    const bool whole = a.ids == nullptr;

    wait_for_predecessor();
    const Row row = row_of(a, b);
    const int64_t row_base = int64_t(b) * a.row_cap;
    if (!whole && a.n_ids_out != nullptr && part == 0 && kvh == 0 && tid == 0) a.n_ids_out[b] = __ldcg(a.n_ids + b);
    if (!row.ok) {  // the merge writes the zeros
        if (part == 0 && kvh == 0 && tid == 0) set_error(a.err, row.t_ok ? QSA_DEVERR_ROW_RANGE : QSA_DEVERR_VISIBLE_RANGE);
        return;
    }
    const int per_run = coded_run_groups(row.groups, whole);
    const int runs = (row.groups + per_run - 1) / per_run;
    if (part >= runs + (row.tail > 0 ? 1 : 0)) return;
    const int64_t pbase = (int64_t(b) * a.q_heads + h0) * a.nparts + part;  // head h0, this run

    if (part == runs) {
        // ---- the raw tail: at most 3 tokens, a warp per head ------------------------
        if (tid < row.tail) {
            const int id = whole ? kGroup * row.groups + tid : __ldcg(a.ids + row_base + kGroup * row.groups + tid);
            if (!whole && kvh == 0 && a.ids_out != nullptr) a.ids_out[row_base + kGroup * row.groups + tid] = id;
            int slot = -1;
            if (id < 0 || id >= row.T) {
                set_error(a.err, QSA_DEVERR_ROW_RANGE);
            } else {
                slot = __ldg(a.slot_map + __ldg(a.slot_offset + b) + id);
                if (slot < 0 || slot >= a.num_slots) {
                    set_error(a.err, QSA_DEVERR_SLOT_RANGE);
                    slot = -1;
                }
            }
            sm.traw[tid] = slot;
        }
        __syncthreads();
        constexpr int kPer = D / 32;
        for (int h = warp; h < gq; h += kWarps) {
            const float *q = a.q + (int64_t(b) * a.q_heads + h0 + h) * D;
            float x[3] = {-INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int t = 0; t < 3; ++t) {
                if (t >= row.tail) continue;
                float dot = 0.0f;
                if (sm.traw[t] >= 0) {
                    const float *k = a.k_cache + (int64_t(sm.traw[t]) * a.kv_heads + kvh) * D;
#pragma unroll
                    for (int j = 0; j < kPer; ++j) dot = fmaf(__ldg(q + lane + 32 * j), __ldg(k + lane + 32 * j), dot);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
                x[t] = dot * (a.scale * kLog2e);
            }
            const float m = fmaxf(fmaxf(x[0], x[1]), x[2]);
            const float ms = m == -INFINITY ? 0.0f : m;
            float p[3], l = 0.0f;
#pragma unroll
            for (int t = 0; t < 3; ++t) {
                p[t] = t < row.tail ? ex2(x[t] - ms) : 0.0f;
                l += p[t];
            }
            float *acc = a.part_acc + (pbase + int64_t(h) * a.nparts) * D;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                float o = 0.0f;
#pragma unroll
                for (int t = 0; t < 3; ++t) {
                    if (t >= row.tail || sm.traw[t] < 0) continue;
                    o = fmaf(p[t], __ldg(a.v_cache + (int64_t(sm.traw[t]) * a.kv_heads + kvh) * D + lane + 32 * j), o);
                }
                acc[lane + 32 * j] = o;
            }
            if (lane == 0) {
                a.part_m[pbase + int64_t(h) * a.nparts] = m;
                a.part_l[pbase + int64_t(h) * a.nparts] = l;
            }
        }
        return;
    }

    const int run_end = min(row.groups, (part + 1) * per_run);
    const int32_t *bmap = a.block_map + __ldg(a.block_offset + b);
    // thread t takes group seg + t: its block first, so that copies can start, ...
    auto resolve_block = [&](int seg) {
        if (tid >= kSegGroups) return -1;
        int blk = -1;
        if (tid < min(kSegGroups, run_end - seg)) {
            int g = seg + tid;
            bool good = true;
            if (!whole) {
                const int32_t *ids = a.ids + row_base + kGroup * int64_t(g);
                int id[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) id[u] = __ldcg(ids + u);
                if (kvh == 0 && a.ids_out != nullptr) {
#pragma unroll
                    for (int u = 0; u < 4; ++u) a.ids_out[row_base + kGroup * int64_t(g) + u] = id[u];
                }
                good = id[0] >= 0 && id[0] % kGroup == 0 && id[0] <= row.T - kGroup && id[1] == id[0] + 1 &&
                       id[2] == id[0] + 2 && id[3] == id[0] + 3;
                g = id[0] / kGroup;
                if (!good) set_error(a.err, QSA_DEVERR_ROW_RANGE);
            }
            blk = -2;
            if (good) {
                blk = __ldg(bmap + g);
                if (blk < 0 || blk >= a.num_blocks) {
                    blk = -2;
                    set_error(a.err, QSA_DEVERR_SLOT_RANGE);
                }
            }
        }
        sm.blk[tid] = blk;
        return blk;
    };
    // ... then its scales, the V scales of a step's 4 groups brought to a common power of two
    auto load_scales = [&](int blk) {
        return blk >= 0 ? __ldg(reinterpret_cast<const float2 *>(a.scales) + int64_t(blk) * a.kv_heads + kvh)
                        : make_float2(0.0f, 0.0f);
    };
    auto store_meta = [&](int blk, float2 sc) {
        if (tid >= kSegGroups) return;
        uint32_t top = __float_as_uint(sc.y) & 0x7fffffffu;
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        float f, inv;
        scale_to<kVTop>(top, f, inv);
        sm.meta[tid] = make_float4(sc.x, sc.y * f, inv, blk != -1 ? 1.0f : 0.0f);
    };
    const unsigned char *codes = a.codes + int64_t(kvh) * (8 * D);
    const int64_t blk_bytes = int64_t(a.kv_heads) * (8 * D);
    auto issue = [&](int g0, int slot) {  // the step at group g0 of the segment: lane u < 4 copies group u
        unsigned char *dst = sm.ring[warp][slot];
        uint64_t *bar = &sm.full[warp][slot];
        const int blk = lane < kStepGroups ? sm.blk[g0 + lane] : -1;
        const uint32_t there = __ballot_sync(0xffffffffu, blk >= 0);
        if (lane == 0) {
            if (there != 0) mbar_arrive_expect_tx(bar, uint32_t(__popc(there)) * (8 * D));
            else mbar_arrive(bar);
        }
        __syncwarp();
        if (blk >= 0) bulk_copy_g2s(dst + lane * S::kBlk, codes + blk * blk_bytes, 8 * D, bar);
        if (there != (1u << kStepGroups) - 1u) {  // groups that are not there, or not to be read: zeros
            for (int u = 0; u < kStepGroups; ++u) {
                if ((there >> u) & 1u) continue;
                for (int c = lane; c < 8 * D / 16; c += 32)
                    *reinterpret_cast<uint4 *>(dst + u * S::kBlk + c * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();  // a later step copies into these bytes
        }
    };
    if (tid < kWarps * kRing) mbar_init(&sm.full[0][0] + tid, 1);
    fence_mbar_init();
    int my_blk = resolve_block(part * per_run);
    __syncthreads();
    // this warp's steps of the segment in hand: groups g0 = 4 * (warp + kWarps * k)
    auto steps_of = [&](int seg) {
        const int n = (min(kSegGroups, run_end - seg) + kStepGroups - 1) / kStepGroups;
        return n > warp ? (n - warp + kWarps - 1) / kWarps : 0;
    };
    int my_steps = steps_of(part * per_run);
    int in_slot = 0;                       // the ring slot of the next step to issue
    auto issue_next = [&](int k) {
        issue((warp + kWarps * k) * kStepGroups, in_slot);
        in_slot = in_slot == kRing - 1 ? 0 : in_slot + 1;
    };
#pragma unroll
    for (int k = 0; k < kRing - 1; ++k)
        if (k < my_steps) issue_next(k);
    const float2 my_scales = load_scales(my_blk);

    // ---- the queries: the matrix operands of each 16 dims, hi and lo ---------------------
    // hi and lo words of dims 4u..4u+3 of the 16 that lane (head hl + 8*s, i4) holds of
    // half j, with the head's power of two taken out
    auto q_scale = [&](int s, float &f, float &inv) {
        uint32_t top = 0;
        const int h = hl + 8 * s;
        if (h < gq) {
            const float4 *src = reinterpret_cast<const float4 *>(a.q + (int64_t(b) * a.q_heads + h0 + h) * D + 16 * i4);
#pragma unroll
            for (int j = 0; j < kHalves; ++j)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float4 x = __ldg(src + 16 * j + u);
                    top = max(top, max(__float_as_uint(x.x) & 0x7fffffffu, __float_as_uint(x.y) & 0x7fffffffu));
                    top = max(top, max(__float_as_uint(x.z) & 0x7fffffffu, __float_as_uint(x.w) & 0x7fffffffu));
                }
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        scale_to<kQTop>(top, f, inv);
    };
    auto q_words = [&](int s, int j, int u, float f, uint32_t (&hi)[2], uint32_t (&lo)[2]) {
        const int h = hl + 8 * s;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (h < gq)
            x = __ldg(reinterpret_cast<const float4 *>(a.q + (int64_t(b) * a.q_heads + h0 + h) * D + 64 * j + 16 * i4) + u);
        split2(x.x * f, x.y * f, hi[0], lo[0]);
        split2(x.z * f, x.w * f, hi[1], lo[1]);
    };
    uint32_t qa[HS == 1 ? kHalves : 1][4][4];  // (up to 8 heads: in registers)
    float hscale[HS], qf[HS];
#pragma unroll
    for (int s = 0; s < HS; ++s) {
        float inv;
        q_scale(s, qf[s], inv);
        hscale[s] = a.scale * kLog2e * inv;
    }
    if constexpr (HS == 1) {
#pragma unroll
        for (int j = 0; j < kHalves; ++j)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                uint32_t hi[2], lo[2];
                q_words(0, j, u, qf[0], hi, lo);
                qa[j][u][0] = hi[0];
                qa[j][u][1] = lo[0];
                qa[j][u][2] = hi[1];
                qa[j][u][3] = lo[1];
            }
    } else {
        for (int e = warp; e < kHalves * 4; e += kWarps) {
            uint32_t hi[2][2], lo[2][2];
#pragma unroll
            for (int s = 0; s < 2; ++s) q_words(s, e / 4, e % 4, qf[s], hi[s], lo[s]);
            sm.qa[e][0][lane] = make_uint4(hi[0][0], hi[1][0], hi[0][1], hi[1][1]);
            sm.qa[e][1][lane] = make_uint4(lo[0][0], lo[1][0], lo[0][1], lo[1][1]);
        }
    }

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

    store_meta(my_blk, my_scales);
    __syncthreads();

    int slot = 0;                          // of the step in hand, and the phase of its barrier
    uint32_t phase = 0;
    bool timed_out = false;
    for (int seg = part * per_run; seg < run_end; seg += kSegGroups) {
        if (seg != part * per_run) {       // (rows beyond 65,536 groups: runs of several segments)
            my_blk = resolve_block(seg);
            store_meta(my_blk, load_scales(my_blk));
            __syncthreads();
            my_steps = timed_out ? 0 : steps_of(seg);
#pragma unroll
            for (int k = 0; k < kRing - 1; ++k)
                if (k < my_steps) issue_next(k);
        }
        for (int k = 0; k < my_steps; ++k) {
            if (k + kRing - 1 < my_steps) issue_next(k + kRing - 1);  // into the slot that step k-1 used
            if (!mbar_wait_bounded(&sm.full[warp][slot], phase, kWaitLimitNs)) {
                timed_out = true;
                if (lane == 0) set_error(a.err, QSA_DEVERR_WAIT_TIMEOUT);
                for (int o = k + 1; o < min(my_steps, k + kRing); ++o) {  // let the copies in flight land
                    if (++slot == kRing) slot = 0, phase ^= 1u;
                    (void)mbar_wait_bounded(&sm.full[warp][slot], phase, kDrainLimitNs);
                }
                break;
            }
            __syncwarp();
            const unsigned char *blk0 = sm.ring[warp][slot];
            const int g0 = (warp + kWarps * k) * kStepGroups;
            const float4 meta = sm.meta[g0 + i4];

            // ---- scores of the step's 16 tokens: two tiles of 8 ---------------------------
            float x[HS][4];
            {
                float c[2][kHalves][4];  // a chain of 4 (9 to 16 heads: 8) per tile and half
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
                                if (u == 0) mma16816_first(c[t][j], qa[j][u], b0, b1);
                                else mma16816(c[t][j], qa[j][u], b0, b1);
                            } else {
                                if (u == 0) mma16816_first(c[t][j], qh, b0, b1);
                                else mma16816(c[t][j], qh, b0, b1);
                                mma16816(c[t][j], ql, b0, b1);
                            }
                        }
                    }
                }
                // rows hl and hl+8 are the hi and lo parts of a head, or two heads
#pragma unroll
                for (int s = 0; s < HS; ++s) {
                    const float f = hscale[s] * meta.x;
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            float v = HS == 1 ? c[t][0][u] + c[t][0][u + 2] : c[t][0][u + 2 * s];
#pragma unroll
                            for (int j = 1; j < kHalves; ++j)
                                v += HS == 1 ? c[t][j][u] + c[t][j][u + 2] : c[t][j][u + 2 * s];
                            x[s][2 * t + u] = meta.w != 0.0f ? v * f : -INFINITY;
                        }
                }
            }

            // ---- softmax of this lane's heads over the step, relative to m_run ----------------
            // m_run follows the largest score only when that passes it by more than
            // 2^kLag, so that the accumulators are rescaled a few times in a row and
            // not at almost every step; weights stay below 2^kLag.
            uint32_t ph[HS][2], pl[HS][2];
            float mc[HS];
            bool passed = false;
#pragma unroll
            for (int s = 0; s < HS; ++s) {
                mc[s] = fmaxf(fmaxf(x[s][0], x[s][1]), fmaxf(x[s][2], x[s][3]));
                mc[s] = fmaxf(mc[s], __shfl_xor_sync(0xffffffffu, mc[s], 1));
                mc[s] = fmaxf(mc[s], __shfl_xor_sync(0xffffffffu, mc[s], 2));
                passed = passed || mc[s] > m_run[s] + float(kLag);
            }
            if (__any_sync(0xffffffffu, passed)) {
#pragma unroll
                for (int s = 0; s < HS; ++s) {
                    if (!(mc[s] > m_run[s] + float(kLag))) mc[s] = m_run[s];
                    const float alpha = mc[s] == -INFINITY ? 1.0f : ex2(m_run[s] - mc[s]);
                    m_run[s] = mc[s];
                    l_run[s] *= alpha;
#pragma unroll
                    for (int j = 0; j < kVC; ++j)
#pragma unroll
                        for (int u = 0; u < 4; ++u) acc[s][j][u] = mul2(acc[s][j][u], alpha);
                }
            }
#pragma unroll
            for (int s = 0; s < HS; ++s) {
                const float ms = m_run[s] == -INFINITY ? 0.0f : m_run[s];
                float p[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) p[u] = ex2(x[s][u] - ms);
                const float gs = (p[0] + p[1]) + (p[2] + p[3]);
                l_run[s] += gs;
                split2(p[0] * meta.y, p[1] * meta.y, ph[s][0], pl[s][0]);
                split2(p[2] * meta.y, p[3] * meta.y, ph[s][1], pl[s][1]);
                const int h = hl + 8 * s;
                if (a.mass != nullptr && h < gq) {
                    const int64_t hb = int64_t(b) * a.q_heads + h0 + h;
                    if (meta.w != 0.0f) a.mass[hb * a.mass_stride + seg + g0 + i4] = gs;
                    if (i4 == 0) a.mref[hb * (a.mass_stride / 4) + (seg + g0) / 4] = ms;
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
                        acc[0][j][u] = fma2(add2(make_float2(c[0], c[1]), make_float2(c[2], c[3])), meta.z, acc[0][j][u]);
                    } else {
                        mma16816(c, pb, b0, b1);
                        acc[0][j][u] = fma2(make_float2(c[0], c[1]), meta.z, acc[0][j][u]);
                        acc[HS - 1][j][u] = fma2(make_float2(c[2], c[3]), meta.z, acc[HS - 1][j][u]);
                    }
                }
            }
            __syncwarp();  // the slot is refilled by a later step
            if (++slot == kRing) slot = 0, phase ^= 1u;
        }
        __syncthreads();  // every warp is done with the segment's blocks and ring
    }

    // ---- this run's state: the warps' states merged in warp order -----------------------
    float *red = reinterpret_cast<float *>(sm.ring);  // [kWarps][kNH][D]
#pragma unroll
    for (int s = 0; s < HS; ++s) {
        const int h = hl + 8 * s;
#pragma unroll
        for (int j = 0; j < kVC; ++j) {
            float4 *dst = reinterpret_cast<float4 *>(red + (warp * kNH + h) * D + 32 * j + 8 * i4);
            dst[0] = make_float4(acc[s][j][0].x, acc[s][j][1].x, acc[s][j][2].x, acc[s][j][3].x);
            dst[1] = make_float4(acc[s][j][0].y, acc[s][j][1].y, acc[s][j][2].y, acc[s][j][3].y);
        }
        float l = l_run[s];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (i4 == 0) {
            sm.wm[warp][h] = m_run[s];
            sm.wl[warp][h] = l;
        }
    }
    __syncthreads();
    if (tid < gq) {
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.wm[w][tid]);
        const float Ms = M == -INFINITY ? 0.0f : M;
        float L = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float wt = ex2(sm.wm[w][tid] - Ms);
            sm.ww[w][tid] = wt;
            L = fmaf(sm.wl[w][tid], wt, L);
        }
        a.part_m[pbase + int64_t(tid) * a.nparts] = M;
        a.part_l[pbase + int64_t(tid) * a.nparts] = L;
    }
    __syncthreads();
    constexpr int F4 = D / 4;
    for (int e = tid; e < gq * F4; e += kThreads) {
        const int h = e / F4, c = e % F4;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float4 p = *reinterpret_cast<const float4 *>(red + (w * kNH + h) * D + 4 * c);
            const float wt = sm.ww[w][h];
            o.x = fmaf(p.x, wt, o.x);
            o.y = fmaf(p.y, wt, o.y);
            o.z = fmaf(p.z, wt, o.z);
            o.w = fmaf(p.w, wt, o.w);
        }
        reinterpret_cast<float4 *>(a.part_acc + (pbase + int64_t(h) * a.nparts) * D)[c] = o;
    }
}

// ---- the runs of a row merged in run order ---------------------------------------------
// One CTA per (head, query): M = max m_c, w_c = 2^(m_c - M), L = sum l_c w_c,
// out = sum acc_c w_c / L.  Eight slices of threads take the runs c = s, s+8, ..
// and their sums are added in slice order.
constexpr int kMergeThreads = 256;
constexpr int kMaxRuns = 514;
// of AttendCodedArgs::sharing
constexpr uint32_t kBad = 1u, kFirstSharer = 2u, kLaterSharer = 4u;

// Whether query b's row may add weights, and to whose accumulators; a CTA of its
// own beside the merge's.
__device__ void find_sharing(const AttendCodedArgs &a, int b, const Row &row)
{
    const int tid = threadIdx.x;
    const bool whole = a.ids == nullptr;
    // its groups are well formed and ascend
    int bad = row.ok ? 0 : 1;
    if (!whole && row.ok) {
        const int32_t *ids = a.ids + int64_t(b) * a.row_cap;
        for (int g = tid; g < row.groups; g += kMergeThreads) {
            int id[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) id[u] = __ldcg(ids + kGroup * g + u);
            const bool good = id[0] >= 0 && id[0] % kGroup == 0 && id[0] <= row.T - kGroup && id[1] == id[0] + 1 &&
                              id[2] == id[0] + 2 && id[3] == id[0] + 3 && (g == 0 || __ldcg(ids + kGroup * g - 4) < id[0]);
            if (!good) bad = 1;
        }
        for (int j = tid; j < row.tail; j += kMergeThreads) {
            const int id = __ldcg(ids + kGroup * row.groups + j);
            if (id < 0 || id >= row.T || id / kGroup != row.T / kGroup) bad = 1;
        }
    }
    bad = __syncthreads_or(bad);
    // and whose accumulators it adds to: its own, or those of several queries
    const int64_t off = __ldg(a.weight_offset + b);
    int earlier = 0, later = 0;
    for (int o = tid; o < a.batch; o += kMergeThreads) {
        if (o != b && __ldg(a.weight_offset + o) == off) (o < b ? earlier : later) = 1;
    }
    earlier = __syncthreads_or(earlier);
    later = __syncthreads_or(later);
    if (!whole && (earlier || later) && !bad) {  // its row of shares: nothing for the groups that it does not name
        float4 *map = reinterpret_cast<float4 *>(a.share_map + int64_t(b) * a.map_stride);
        for (int g = tid; g < a.map_stride / 4; g += kMergeThreads) map[g] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (tid == 0) {
        a.sharing[b] = (bad ? kBad : 0u) | (earlier ? kLaterSharer : later ? kFirstSharer : 0u);
        if (bad && row.ok) set_error(a.err, QSA_DEVERR_ROW_RANGE);
    }
}

template <int D>
__global__ void __launch_bounds__(kMergeThreads) merge_coded_kernel(const AttendCodedArgs a)
{
    constexpr int F4 = D / 4;
    constexpr int kSlices = kMergeThreads / F4;
    __shared__ float w[kMaxRuns];
    __shared__ float red[kMergeThreads / 32];
    __shared__ float s_m, s_l;
    __shared__ float4 part[kSlices][F4];
    const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    wait_for_predecessor();
    const bool whole = a.ids == nullptr;
    const Row row = row_of(a, b);
    if (h == a.q_heads) {
        find_sharing(a, b, row);
        return;
    }
    const int per_run = coded_run_groups(row.groups, whole);
    const int used = (row.groups + per_run - 1) / per_run + (row.tail > 0 ? 1 : 0);
    const int64_t hb = int64_t(b) * a.q_heads + h;
    const float *pm = a.part_m + hb * a.nparts, *pl = a.part_l + hb * a.nparts;

    float m = -INFINITY;
    for (int c = tid; c < used; c += kMergeThreads) m = fmaxf(m, __ldcg(pm + c));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((tid & 31) == 0) red[tid >> 5] = m;
    __syncthreads();
    if (tid == 0) {
        float M = -INFINITY;
        for (int k = 0; k < kMergeThreads / 32; ++k) M = fmaxf(M, red[k]);
        s_m = M == -INFINITY ? 0.0f : M;
    }
    __syncthreads();
    const float M = s_m;
    float l = 0.0f;
    for (int c = tid; c < used; c += kMergeThreads) {
        const float wt = ex2(__ldcg(pm + c) - M);
        w[c] = wt;
        l = fmaf(__ldcg(pl + c), wt, l);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if ((tid & 31) == 0) red[tid >> 5] = l;
    __syncthreads();
    if (tid == 0) {
        float L = 0.0f;
        for (int k = 0; k < kMergeThreads / 32; ++k) L += red[k];
        s_l = L;
        if (a.stat != nullptr) {
            a.stat[2 * hb] = M;
            a.stat[2 * hb + 1] = L > 0.0f || L != L ? 1.0f / L : 0.0f;
        }
    }
    // columns
    const int col = tid % F4, slice = tid / F4;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = slice; c < used; c += kSlices) {
        const float4 x = __ldcg(reinterpret_cast<const float4 *>(a.part_acc + (hb * a.nparts + c) * D) + col);
        const float wt = w[c];
        o.x = fmaf(x.x, wt, o.x);
        o.y = fmaf(x.y, wt, o.y);
        o.z = fmaf(x.z, wt, o.z);
        o.w = fmaf(x.w, wt, o.w);
    }
    part[slice][col] = o;
    __syncthreads();
    if (slice == 0) {
        const float L = s_l;
#pragma unroll
        for (int k = 1; k < kSlices; ++k) {
            const float4 x = part[k][col];
            o.x += x.x;
            o.y += x.y;
            o.z += x.z;
            o.w += x.w;
        }
        // L = 0: no token (or none above -inf); a NaN denominator gives NaN
        float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
        if (L > 0.0f || L != L) r = make_float4(o.x / L, o.y / L, o.z / L, o.w / L);
        reinterpret_cast<float4 *>(a.out + hb * D)[col] = r;
    }
}

// ---- the groups' shares of attention added to the accumulators --------------------------
// weights[weight_offset[b] + g] += sum_h share(b, h, g), share = mass * 2^(mref - M_h) / L_h.
// No atomics: a query with accumulators of its own adds its shares as they come
// (own_weights_kernel); queries that share them are added in a fixed order, eight
// threads per group (shared_weights_kernel), so that the sum has one value.
// Selected rows of such queries are first spread out to one share per group of
// the history (in the workspace's scores, which nobody needs by then), so that
// the second kernel reads rows side by side: on 256 queries that share a history
// of 25,064 groups, searching each group in each query's row instead took 1540 us.
constexpr int kAccThreads = 256;
constexpr int kOwnSlices = 4;                          // threads per position, a quarter of the heads each
constexpr int kOwnPos = kAccThreads / kOwnSlices;
constexpr int kSharedSlices = 8;                       // threads per group, an eighth of the queries each
constexpr int kSharedGroups = kAccThreads / kSharedSlices;

// Heads h0, h0 + step, .. of position pos.
__device__ __forceinline__ float share_of(const AttendCodedArgs &a, int b, int pos, int h0, int step)
{
    float s = 0.0f;
    const int64_t hb = int64_t(b) * a.q_heads;
    const float *mass = a.mass + hb * a.mass_stride + pos;
    const float *mref = a.mref + hb * (a.mass_stride / 4) + pos / 4;
    const float2 *stat = reinterpret_cast<const float2 *>(a.stat) + hb;
#pragma unroll 4
    for (int h = h0; h < a.q_heads; h += step) {
        const float2 st = __ldcg(stat + h);
        const float g = __ldcg(mass + int64_t(h) * a.mass_stride);
        const float r = __ldcg(mref + int64_t(h) * (a.mass_stride / 4));
        s = fmaf(g * ex2(r - st.x), st.y, s);
    }
    return s;
}

// The same of the raw tail: its run's state.
__device__ __forceinline__ float tail_share_of(const AttendCodedArgs &a, int b, int run, int h0, int step)
{
    float s = 0.0f;
    const int64_t hb = int64_t(b) * a.q_heads;
    const float2 *stat = reinterpret_cast<const float2 *>(a.stat) + hb;
#pragma unroll 4
    for (int h = h0; h < a.q_heads; h += step) {
        const float2 st = __ldcg(stat + h);
        const int64_t at = (hb + h) * a.nparts + run;
        s = fmaf(__ldcg(a.part_l + at) * ex2(__ldcg(a.part_m + at) - st.x), st.y, s);
    }
    return s;
}

__device__ __forceinline__ int tail_run(const Row &row, bool whole)
{
    const int per = coded_run_groups(row.groups, whole);
    return (row.groups + per - 1) / per;
}

__global__ void __launch_bounds__(kAccThreads) own_weights_kernel(const AttendCodedArgs a)
{
    __shared__ float sum[kOwnSlices][kOwnPos];
    const int b = blockIdx.y, lp = threadIdx.x % kOwnPos, slice = threadIdx.x / kOwnPos;
    const bool whole = a.ids == nullptr;
    wait_for_predecessor();
    const uint32_t sharing = __ldcg(a.sharing + b);
    const Row row = row_of(a, b);
    if (sharing & kBad) return;
    const bool own = sharing == 0;
    // (shared accumulators of whole histories: shared_weights_kernel reads the masses itself)
    const int first = !own && whole ? row.groups : 0, end = row.groups + (row.tail > 0 ? 1 : 0);
    for (int64_t p0 = first + int64_t(blockIdx.x) * kOwnPos; p0 < end; p0 += int64_t(gridDim.x) * kOwnPos) {
        const int p = int(p0) + lp;
        int g = row.T / kGroup;
        if (slice == 0 && p < row.groups) g = whole ? p : __ldcg(a.ids + int64_t(b) * a.row_cap + kGroup * p) / kGroup;
        float s = 0.0f;
        if (p < row.groups) s = share_of(a, b, p, slice, kOwnSlices);
        else if (p < end) s = tail_share_of(a, b, tail_run(row, whole), slice, kOwnSlices);
        sum[slice][lp] = s;
        __syncthreads();
        if (slice == 0 && p < end) {
#pragma unroll
            for (int k = 1; k < kOwnSlices; ++k) s += sum[k][lp];
            if (own) a.weights[__ldg(a.weight_offset + b) + g] += s;
            else if (p == row.groups) a.tail_share[b] = s;
            else a.share_map[int64_t(b) * a.map_stride + g] = s;
        }
        __syncthreads();
    }
}

template <bool kWhole>
__global__ void __launch_bounds__(kAccThreads) shared_weights_kernel(const AttendCodedArgs a)
{
    __shared__ int2 member[kAccThreads];  // per query: complete groups of its history (-1: adds nothing here), tail
    __shared__ float sum[kSharedSlices][kSharedGroups];
    __shared__ uint32_t first_of[kAccThreads / 32];
    constexpr int kAhead = 8;             // shares loaded before they are added
    const int tid = threadIdx.x, lg = tid % kSharedGroups, slice = tid / kSharedGroups;
    const int groups = a.max_visible / kGroup + 1;
    wait_for_predecessor();
    for (int b0 = 0; b0 < a.batch; b0 += kAccThreads) {
        const bool first = b0 + tid < a.batch && (__ldcg(a.sharing + b0 + tid) & kFirstSharer);
        const uint32_t firsts = __ballot_sync(0xffffffffu, first);
        if (!__syncthreads_or(first)) continue;
        if (tid % 32 == 0) first_of[tid / 32] = firsts;
        __syncthreads();
        for (int i = 0; i < kAccThreads; ++i) {  // the histories' first queries
            const uint32_t left = first_of[i / 32] >> (i % 32);
            if (left == 0) {  // none in the rest of the 32
                i |= 31;
                continue;
            }
            i += __ffs(left) - 1;
            const int b = b0 + i;
            const int64_t off = __ldg(a.weight_offset + b);
            for (int64_t g0 = int64_t(blockIdx.x) * kSharedGroups; g0 < groups; g0 += int64_t(gridDim.x) * kSharedGroups) {
                const int g = int(g0) + lg;
                float s = 0.0f;
                for (int o0 = b; o0 < a.batch; o0 += kAccThreads) {
                    const int n = min(kAccThreads, a.batch - o0);
                    __syncthreads();
                    member[tid] = make_int2(-1, 0);
                    if (tid < n && __ldg(a.weight_offset + o0 + tid) == off && !(__ldcg(a.sharing + o0 + tid) & kBad)) {
                        const Row row = row_of(a, o0 + tid);
                        member[tid] = make_int2(row.T / kGroup, row.tail);
                    }
                    __syncthreads();
                    if constexpr (kWhole) {
                        for (int j = slice; j < n; j += kSharedSlices)
                            if (g < member[j].x) s += share_of(a, o0 + j, g, 0, 1);
                    } else {
                        for (int j = slice; j < n; j += kSharedSlices * kAhead) {
                            float t[kAhead];
#pragma unroll
                            for (int u = 0; u < kAhead; ++u) {
                                const int o = min(j + u * kSharedSlices, n - 1);  // (every load is made, no branch between them)
                                t[u] = __ldcg(a.share_map + int64_t(o0 + o) * a.map_stride + min(g, a.map_stride - 1));
                            }
#pragma unroll
                            for (int u = 0; u < kAhead; ++u) {
                                const int o = j + u * kSharedSlices;
                                if (o < n && g < member[o].x) s += t[u];
                            }
                        }
                    }
                    for (int j = slice; j < n; j += kSharedSlices)  // the raw tails
                        if (member[j].x == g && member[j].y > 0) s += __ldcg(a.tail_share + o0 + j);
                }
                sum[slice][lg] = s;
                __syncthreads();
                if (slice == 0) {
#pragma unroll
                    for (int k = 1; k < kSharedSlices; ++k) s += sum[k][lg];
                    if (s != 0.0f) a.weights[off + g] += s;
                }
                __syncthreads();
            }
        }
        __syncthreads();  // first_of is filled again
    }
}

template <int D, int HS, bool kInt8>
cudaError_t launch_t(const AttendCodedArgs &a, int runs, cudaStream_t s, bool pdl)
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
    return launch_kernel(attend_coded_kernel<D, HS, kInt8>, dim3(unsigned(runs), unsigned(a.kv_heads), unsigned(a.batch)),
                         dim3(kThreads), smem, s, pdl, a);
}

static_assert(sizeof(Sm<128, 2>) <= 227 * 1024, "shared memory per CTA");
static_assert(4 * (sizeof(Sm<128, 1>) + 1024) <= 228 * 1024, "four CTAs per SM with one head set");
static_assert(kThreads >= kSegGroups, "a thread resolves a group");
static_assert(kWarps * 16 * 128 * 4 <= int(sizeof(Sm<128, 2>::ring)) && kWarps * 16 * 64 * 4 <= int(sizeof(Sm<64, 2>::ring)),
              "the reduction area fits the ring");

}  // namespace

bool attend_coded_shape_supported(int head_dim, int q_heads, int kv_heads)
{
    return (head_dim == 64 || head_dim == 128) && q_heads / kv_heads <= kMaxGqa && kv_heads <= 65535 && q_heads <= 65535;
}

cudaError_t launch_attend_coded(const AttendCodedArgs &a, cudaStream_t s, bool pdl)
{
    if (a.batch == 0) return cudaSuccess;
    const bool whole = a.ids == nullptr;
    const int runs = whole ? coded_max_runs(a.max_visible / kGroup, true) : coded_max_runs((a.row_cap - 3) / kGroup, false);
    const bool one = a.q_heads / a.kv_heads <= 8, i8 = a.format == QSA_CODE_INT8;
    cudaError_t e;
    if (a.head_dim == 128)
        e = one ? (i8 ? launch_t<128, 1, true>(a, runs, s, pdl) : launch_t<128, 1, false>(a, runs, s, pdl))
                : (i8 ? launch_t<128, 2, true>(a, runs, s, pdl) : launch_t<128, 2, false>(a, runs, s, pdl));
    else
        e = one ? (i8 ? launch_t<64, 1, true>(a, runs, s, pdl) : launch_t<64, 1, false>(a, runs, s, pdl))
                : (i8 ? launch_t<64, 2, true>(a, runs, s, pdl) : launch_t<64, 2, false>(a, runs, s, pdl));
    if (e != cudaSuccess) return e;
    const dim3 mgrid(unsigned(a.q_heads + (a.weights != nullptr ? 1 : 0)), unsigned(a.batch));
    e = a.head_dim == 128 ? launch_kernel(merge_coded_kernel<128>, mgrid, dim3(kMergeThreads), 0, s, true, a)
                          : launch_kernel(merge_coded_kernel<64>, mgrid, dim3(kMergeThreads), 0, s, true, a);
    if (e != cudaSuccess || a.weights == nullptr) return e;
    const int positions = (whole ? a.max_visible : a.row_cap) / kGroup + 1;
    const int blocks = (positions + kOwnPos - 1) / kOwnPos;
    e = launch_kernel(own_weights_kernel, dim3(unsigned(blocks < 1024 ? blocks : 1024), unsigned(a.batch)), dim3(kAccThreads), 0,
                      s, true, a);
    if (e != cudaSuccess || a.batch == 1) return e;
    const int shared_blocks = (a.max_visible / kGroup + kSharedGroups) / kSharedGroups;
    return launch_kernel(whole ? shared_weights_kernel<true> : shared_weights_kernel<false>,
                         dim3(unsigned(shared_blocks < 1024 ? shared_blocks : 1024)), dim3(kAccThreads), 0, s, true, a);
}

}  // namespace qsa
