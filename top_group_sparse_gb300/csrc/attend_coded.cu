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
// two sets.)  Every instruction chain starts from zero and its result is added
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

constexpr int kWarps = 8;
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
    int blk[kSegGroups];                                     // physical block; -1: none, -2: zero rows
    float wm[kWarps][8 * HS], wl[kWarps][8 * HS], ww[kWarps][8 * HS];
    float tx[8 * HS][4];
    int traw[4];
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float ex2(float x)
{
    return exp2f(x);
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// Powers of two that bring a largest magnitude (its bits) to [2^13, 2^14), and
// back.  The exponent is kept to -110..128, so that both are normal floats.
__device__ __forceinline__ void scale_to_2_14(uint32_t top, float &f, float &inv)
{
    const int e = max(int(top >> 23) - 127, -110);
    f = __uint_as_float(uint32_t(13 - e + 127) << 23);
    inv = __uint_as_float(uint32_t(e - 13 + 127) << 23);
}

// Length of query b's row, and whether it may be read.
struct Row {
    int groups, tail;   // complete groups; raw tokens behind them
    int T;              // visible tokens
    bool ok;
};
__device__ __forceinline__ Row row_of(const AttendCodedArgs &a, int b)
{
    Row r;
    r.T = __ldg(a.visible + b);
    const int n = a.ids != nullptr ? __ldcg(a.n_ids + b) : r.T;
    r.ok = a.ids != nullptr ? (n >= 0 && n <= a.row_cap) : (n >= 0 && n <= a.max_visible);
    r.groups = r.ok ? n / kGroup : 0;
    r.tail = r.ok ? n % kGroup : 0;
    return r;
}

template <int D, int HS, bool kInt8>
__global__ void __launch_bounds__(kThreads, HS == 1 ? 2 : 1) attend_coded_kernel(const AttendCodedArgs a)
{
    extern __shared__ __align__(128) unsigned char smem_raw[];
    using S = Sm<D, HS>;
    S &sm = *reinterpret_cast<S *>(smem_raw);
    constexpr int kNH = 8 * HS;
    constexpr int kChunks = 8 * D / 16;   // 16-byte pieces of a block
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
        if (part == 0 && kvh == 0 && tid == 0) set_error(a.err, whole ? QSA_DEVERR_VISIBLE_RANGE : QSA_DEVERR_ROW_RANGE);
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

    // ---- the queries: this lane's dims of its head, hi and lo, per set of 8 heads ------
    uint32_t qa[HS][kHalves][4][4];
    float hscale[HS];
#pragma unroll
    for (int s = 0; s < HS; ++s) {
        const int h = hl + 8 * s;
        float v[kHalves][16];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < kHalves; ++j) {
            const float4 *src = reinterpret_cast<const float4 *>(a.q + (int64_t(b) * a.q_heads + h0 + h) * D + 64 * j + 16 * i4);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float4 x = h < gq ? __ldg(src + u) : make_float4(0.f, 0.f, 0.f, 0.f);
                v[j][4 * u] = x.x;
                v[j][4 * u + 1] = x.y;
                v[j][4 * u + 2] = x.z;
                v[j][4 * u + 3] = x.w;
            }
#pragma unroll
            for (int u = 0; u < 16; ++u) top = max(top, __float_as_uint(v[j][u]) & 0x7fffffffu);
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        float f, inv;
        scale_to_2_14(top, f, inv);
        hscale[s] = a.scale * kLog2e * inv;
#pragma unroll
        for (int j = 0; j < kHalves; ++j)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                split2(v[j][4 * u] * f, v[j][4 * u + 1] * f, qa[s][j][u][0], qa[s][j][u][1]);
                split2(v[j][4 * u + 2] * f, v[j][4 * u + 3] * f, qa[s][j][u][2], qa[s][j][u][3]);
            }
    }

    float acc[HS][kVC][8];
    float m_run[HS], l_run[HS];
#pragma unroll
    for (int s = 0; s < HS; ++s) {
        m_run[s] = -INFINITY;
        l_run[s] = 0.0f;
#pragma unroll
        for (int j = 0; j < kVC; ++j)
#pragma unroll
            for (int u = 0; u < 8; ++u) acc[s][j][u] = 0.0f;
    }

    const int run_end = min(row.groups, (part + 1) * per_run);
    const int32_t *bmap = a.block_map + __ldg(a.block_offset + b);
    for (int seg = part * per_run; seg < run_end; seg += kSegGroups) {
        const int n_seg = min(kSegGroups, run_end - seg);
        // ---- resolve: thread t takes group seg + t ---------------------------------------
        if (tid < kSegGroups) {
            int blk = -1;
            float ks = 0.0f, vs = 0.0f;
            if (tid < n_seg) {
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
                if (blk >= 0) {
                    const float2 sc = __ldg(reinterpret_cast<const float2 *>(a.scales) + int64_t(blk) * a.kv_heads + kvh);
                    ks = sc.x;
                    vs = sc.y;
                }
            }
            sm.blk[tid] = blk;
            // the V scales of a step's 4 groups brought to a common power of two
            uint32_t top = __float_as_uint(vs) & 0x7fffffffu;
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            float f, inv;
            scale_to_2_14(top, f, inv);
            sm.meta[tid] = make_float4(ks, vs * f, inv, blk != -1 ? 1.0f : 0.0f);
        }
        __syncthreads();

        const int nsteps = (n_seg + kStepGroups - 1) / kStepGroups;
        const int my_steps = nsteps > warp ? (nsteps - warp + kWarps - 1) / kWarps : 0;
        auto issue = [&](int k) {  // the warp's k-th step of the segment into ring slot k % kRing
            const int g0 = (warp + kWarps * k) * kStepGroups;
            const uint32_t dst = smem_u32(sm.ring[warp][k % kRing]);
#pragma unroll
            for (int e = 0; e < kStepGroups * kChunks / 32; ++e) {
                const int p = e * 32 + lane;
                const int gl = p / kChunks, c = p % kChunks;
                const int blk = sm.blk[g0 + gl];
                if (blk >= 0)
                    cp_async16(dst + gl * S::kBlk + c * 16, a.codes + (int64_t(blk) * a.kv_heads + kvh) * (8 * D) + c * 16);
                else
                    *reinterpret_cast<uint4 *>(sm.ring[warp][k % kRing] + gl * S::kBlk + c * 16) = make_uint4(0, 0, 0, 0);
            }
        };
#pragma unroll
        for (int k = 0; k < kRing - 1; ++k) {
            if (k < my_steps) issue(k);
            cp_async_commit();
        }
        for (int k = 0; k < my_steps; ++k) {
            if (k + kRing - 1 < my_steps) issue(k + kRing - 1);  // into the slot that step k-1 used
            cp_async_commit();
            cp_async_wait<kRing - 1>();
            __syncwarp();
            const unsigned char *blk0 = sm.ring[warp][k % kRing];
            const int g0 = (warp + kWarps * k) * kStepGroups;
            const float4 meta = sm.meta[g0 + i4];

            // ---- scores of the step's 16 tokens: two tiles of 8 ---------------------------
            float x[HS][4];
            {
                float c[HS][2][4];
#pragma unroll
                for (int s = 0; s < HS; ++s)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int u = 0; u < 4; ++u) c[s][t][u] = 0.0f;
                const unsigned char *kp = blk0 + (hl >> 1) * S::kBlk + (hl & 1) * 64 + i4 * 16;
#pragma unroll
                for (int j = 0; j < kHalves; ++j)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(kp + j * 256 + t * 128);
                        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            uint32_t b0, b1;
                            decode4<kInt8>(ww[u], b0, b1);
#pragma unroll
                            for (int s = 0; s < HS; ++s) mma16816(c[s][t], qa[s][j][u], b0, b1);
                        }
                    }
#pragma unroll
                for (int s = 0; s < HS; ++s) {
                    const float f = hscale[s] * meta.x;
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const float v = (c[s][t][u] + c[s][t][u + 2]) * f;
                            x[s][2 * t + u] = meta.w != 0.0f ? v : -INFINITY;
                        }
                }
            }

            // ---- online softmax of this lane's head over the step ---------------------------
            uint32_t pa[HS][4];
            float alpha[HS];
            bool unit = true;
#pragma unroll
            for (int s = 0; s < HS; ++s) {
                float mc = fmaxf(fmaxf(x[s][0], x[s][1]), fmaxf(x[s][2], x[s][3]));
                mc = fmaxf(mc, __shfl_xor_sync(0xffffffffu, mc, 1));
                mc = fmaxf(mc, __shfl_xor_sync(0xffffffffu, mc, 2));
                const float m_new = fmaxf(m_run[s], mc);
                const float ms = m_new == -INFINITY ? 0.0f : m_new;
                alpha[s] = ex2(m_run[s] - ms);
                float p[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) p[u] = ex2(x[s][u] - ms);
                const float gs = (p[0] + p[1]) + (p[2] + p[3]);
                l_run[s] = fmaf(l_run[s], alpha[s], gs);
                m_run[s] = m_new;
                unit = unit && alpha[s] == 1.0f;
                split2(p[0] * meta.y, p[1] * meta.y, pa[s][0], pa[s][1]);
                split2(p[2] * meta.y, p[3] * meta.y, pa[s][2], pa[s][3]);
                const int h = hl + 8 * s;
                if (a.mass != nullptr && h < gq) {
                    const int64_t hb = int64_t(b) * a.q_heads + h0 + h;
                    if (meta.w != 0.0f) a.mass[hb * a.mass_stride + seg + g0 + i4] = gs;
                    if (i4 == 0) a.mref[hb * (a.mass_stride / 4) + (seg + g0) / 4] = ms;
                }
            }
            const bool rescale = !__all_sync(0xffffffffu, unit);

            // ---- weighted values -------------------------------------------------------------
            const unsigned char *vp = blk0 + i4 * S::kBlk + 4 * D + hl * 16;
#pragma unroll
            for (int j = 0; j < kVC; ++j) {
                const uint4 w = *reinterpret_cast<const uint4 *>(vp + j * 128);
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint32_t b0, b1;
                    decode4<kInt8>(ww[u], b0, b1);
#pragma unroll
                    for (int s = 0; s < HS; ++s) {
                        float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        mma16816(c, pa[s], b0, b1);
                        if (rescale) {
                            acc[s][j][u] *= alpha[s];
                            acc[s][j][u + 4] *= alpha[s];
                        }
                        acc[s][j][u] = fmaf(c[0] + c[2], meta.z, acc[s][j][u]);
                        acc[s][j][u + 4] = fmaf(c[1] + c[3], meta.z, acc[s][j][u + 4]);
                    }
                }
            }
            __syncwarp();  // the slot is refilled by a later step
        }
        cp_async_wait<0>();
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
            dst[0] = make_float4(acc[s][j][0], acc[s][j][1], acc[s][j][2], acc[s][j][3]);
            dst[1] = make_float4(acc[s][j][4], acc[s][j][5], acc[s][j][6], acc[s][j][7]);
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
    if (a.bad != nullptr && h == 0) {
        // a row may add weights if its groups are well formed and ascend
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
        if (tid == 0) {
            a.bad[b] = uint32_t(bad);
            if (bad && row.ok) set_error(a.err, QSA_DEVERR_ROW_RANGE);
        }
    }
}

// ---- the groups' shares of attention added to the accumulators --------------------------
// weights[weight_offset[b] + g] += sum_h share(b, h, g),
//   share = mass * 2^(mref - M_h) / L_h.
// The first query of each weight_offset owns its history's row; where other
// queries share it, a thread takes a group and adds their shares in batch order
// (no atomics: the sum has one value).
constexpr int kAccThreads = 256;

__device__ __forceinline__ float share_of(const AttendCodedArgs &a, int b, int pos)
{
    float s = 0.0f;
    for (int h = 0; h < a.q_heads; ++h) {
        const int64_t hb = int64_t(b) * a.q_heads + h;
        const float g = __ldcg(a.mass + hb * a.mass_stride + pos);
        const float r = __ldcg(a.mref + hb * (a.mass_stride / 4) + pos / 4);
        s = fmaf(g * ex2(r - __ldcg(a.stat + 2 * hb)), __ldcg(a.stat + 2 * hb + 1), s);
    }
    return s;
}

// The raw tail's share: its run's state.
__device__ __forceinline__ float tail_share_of(const AttendCodedArgs &a, int b, const Row &row, int run)
{
    float s = 0.0f;
    for (int h = 0; h < a.q_heads; ++h) {
        const int64_t hb = int64_t(b) * a.q_heads + h;
        const float m = __ldcg(a.part_m + hb * a.nparts + run), l = __ldcg(a.part_l + hb * a.nparts + run);
        s = fmaf(l * ex2(m - __ldcg(a.stat + 2 * hb)), __ldcg(a.stat + 2 * hb + 1), s);
    }
    return s;
}

__global__ void __launch_bounds__(kAccThreads) accumulate_kernel(const AttendCodedArgs a)
{
    const int b = blockIdx.y, tid = threadIdx.x;
    wait_for_predecessor();
    const int64_t off = __ldg(a.weight_offset + b);
    bool earlier = false, later = false;
    for (int o = tid; o < a.batch; o += kAccThreads) {
        if (o != b && __ldg(a.weight_offset + o) == off) (o < b ? earlier : later) = true;
    }
    if (__syncthreads_or(earlier)) return;
    const bool shared = __syncthreads_or(later);
    const bool whole = a.ids == nullptr;
    const int64_t first = int64_t(blockIdx.x) * kAccThreads + tid, stride = int64_t(gridDim.x) * kAccThreads;
    float *w = a.weights + off;
    if (!shared) {
        if (__ldcg(a.bad + b)) return;
        const Row row = row_of(a, b);
        const int runs = (row.groups + coded_run_groups(row.groups, whole) - 1) / coded_run_groups(row.groups, whole);
        for (int64_t p = first; p < row.groups + (row.tail > 0 ? 1 : 0); p += stride) {
            if (p == row.groups) {
                w[row.T / kGroup] += tail_share_of(a, b, row, runs);
            } else {
                const int g = whole ? int(p) : __ldcg(a.ids + int64_t(b) * a.row_cap + kGroup * p) / kGroup;
                w[g] += share_of(a, b, int(p));
            }
        }
        return;
    }
    // a shared row: thread per group, the sharing queries in batch order
    for (int64_t g = first; g <= a.max_visible / kGroup; g += stride) {
        float s = 0.0f;
        bool any = false;
        for (int o = b; o < a.batch; ++o) {
            if (__ldg(a.weight_offset + o) != off || __ldcg(a.bad + o)) continue;
            const Row row = row_of(a, o);
            if (row.tail > 0 && g == row.T / kGroup) {
                const int per = coded_run_groups(row.groups, whole);
                const float t = tail_share_of(a, o, row, (row.groups + per - 1) / per);
                s = any ? s + t : w[g] + t;
                any = true;
                continue;
            }
            int pos = -1;
            if (whole) {
                pos = g < row.groups ? int(g) : -1;
            } else {  // the rows ascend
                const int32_t *ids = a.ids + int64_t(o) * a.row_cap;
                int lo = 0, hi = row.groups;
                while (lo < hi) {
                    const int mid = (lo + hi) / 2;
                    if (__ldcg(ids + kGroup * mid) < kGroup * g) lo = mid + 1;
                    else hi = mid;
                }
                if (lo < row.groups && __ldcg(ids + kGroup * lo) == kGroup * g) pos = lo;
            }
            if (pos < 0) continue;
            const float t = share_of(a, o, pos);
            s = any ? s + t : w[g] + t;
            any = true;
        }
        if (any) w[g] = s;
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
static_assert(2 * (sizeof(Sm<128, 1>) + 1024) <= 228 * 1024, "two CTAs per SM with one head set");
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
    const dim3 mgrid(unsigned(a.q_heads), unsigned(a.batch));
    e = a.head_dim == 128 ? launch_kernel(merge_coded_kernel<128>, mgrid, dim3(kMergeThreads), 0, s, true, a)
                          : launch_kernel(merge_coded_kernel<64>, mgrid, dim3(kMergeThreads), 0, s, true, a);
    if (e != cudaSuccess || a.weights == nullptr) return e;
    const int64_t most = a.max_visible / kGroup + 1;
    const int64_t blocks = (most + kAccThreads - 1) / kAccThreads;
    return launch_kernel(accumulate_kernel, dim3(unsigned(blocks < 256 ? blocks : 256), unsigned(a.batch)), dim3(kAccThreads), 0,
                         s, true, a);
}

}  // namespace qsa
