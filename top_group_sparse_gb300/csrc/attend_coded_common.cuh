// attend_coded_common.cuh -- what the attention over 8-bit codes (attend_coded.cu) and that over
// 4-bit ones (attend_coded4.cu) share: a CTA's shape, the operations of a step, and what belongs
// to a query as a whole.
#pragma once

#include <cuda_fp16.h>

#include "cache_internal.cuh"

namespace qsa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

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
// kLog2Units: of what the weights are multiplied with; the inverse makes up for that too.
template <int kLog2Units = 0>
__device__ __forceinline__ void scale_of_weights(float z, float &f, float &inv)
{
    const uint32_t e = __float_as_uint(__fadd_rn(fmaxf(z, -110.0f), 12582912.0f));
    const uint32_t bits = (uint32_t(13 + 127) << 23) - (e << 23);
    f = __uint_as_float(bits);
    inv = __uint_as_float((uint32_t(2 * 127 + kLog2Units) << 23) - bits);
}

constexpr int kLag = 8;     // log2 of the largest softmax weight (16 where the scores' own rounding is that coarse)

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

}  // namespace
}  // namespace qsa
