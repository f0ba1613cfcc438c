// coded.cu -- complete groups' K/V rows turned into 8-bit codes with a scale
// per (group, KV head), for K and for V (include/qsa_cache.h: qsa_code_groups).
//
// s = max|x| * (1/Q) over the group's 4 x d values, code = rn(x / s): each value
// is off by at most half a step of its code's format.  1/Q is the binary32
// number nearest to it and the product and the quotient are correctly rounded,
// so the codes have one value whatever computes them.
//
// Bound by memory: 16*d bytes of K (and of V) read and 4*d written per (group,
// head).  A warp takes one (group, head); a lane holds the same dims of all four
// tokens, so that the V word of a dim (its four tokens) and 16 bytes of V codes
// leave from one lane, and every load is a 16-byte piece of a row.
#include "cache_internal.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Two floats to e4m3 codes, round to nearest even, the lower one first.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

template <bool kInt8>
__device__ __forceinline__ uint32_t code4(float x, float y, float z, float w)
{
    if constexpr (kInt8) {
        auto c = [](float v) { return uint32_t(max(-127, min(127, __float2int_rn(v)))) & 0xffu; };
        return c(x) | (c(y) << 8) | (c(z) << 16) | (c(w) << 24);
    } else {
        return e4m3x2(x, y) | (e4m3x2(z, w) << 16);
    }
}

// Codes the four tokens' rows of K or V of one (group, head), kLanes lanes of 4
// dims each: r[u] are this lane's dims (4*l .. 4*l+3) of token u.  Every lane of
// the warp calls it (two halves may code different rows).
template <int D, bool kInt8>
__device__ __forceinline__ void code_rows(const float4 (&r)[4], int l, bool is_k, uint8_t *dst, float *scale_dst)
{
    uint32_t top = 0;  // bits of the largest |x|: a NaN's are above infinity's, infinity's above every number's
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        top = max(top, __float_as_uint(r[u].x) & 0x7fffffffu);
        top = max(top, __float_as_uint(r[u].y) & 0x7fffffffu);
        top = max(top, __float_as_uint(r[u].z) & 0x7fffffffu);
        top = max(top, __float_as_uint(r[u].w) & 0x7fffffffu);
    }
#pragma unroll
    for (int o = D / 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool finite = top < 0x7f800000u;
    float s = __fmul_rn(__uint_as_float(top), kInt8 ? 1.0f / 127.0f : 1.0f / 448.0f);
    if (s < 1.17549435e-38f) s = 0.0f;  // below the smallest normal float: flushed
    uint32_t c[4] = {0u, 0u, 0u, 0u};
    if (finite && s > 0.0f) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
            c[u] = code4<kInt8>(__fdiv_rn(r[u].x, s), __fdiv_rn(r[u].y, s), __fdiv_rn(r[u].z, s), __fdiv_rn(r[u].w, s));
    }
    if (l == 0) *scale_dst = finite ? s : __int_as_float(0x7fffffff);
    if (is_k) {  // [d/64][4 tokens][64 dims]
#pragma unroll
        for (int u = 0; u < 4; ++u)
            *reinterpret_cast<uint32_t *>(dst + (l / 16) * 256 + u * 64 + (l % 16) * 4) = c[u];
    } else {     // [d][4 tokens]: the 4 x 4 codes transposed
        const uint32_t a = __byte_perm(c[0], c[1], 0x5140), b = __byte_perm(c[2], c[3], 0x5140);
        const uint32_t e = __byte_perm(c[0], c[1], 0x7362), f = __byte_perm(c[2], c[3], 0x7362);
        *reinterpret_cast<uint4 *>(dst + 4 * D + l * 16) =
            make_uint4(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632), __byte_perm(e, f, 0x5410),
                       __byte_perm(e, f, 0x7632));
    }
}

template <int D, bool kInt8>
__global__ void __launch_bounds__(kThreads) code_groups_kernel(const CodeArgs a)
{
    const int b = blockIdx.y;
    const int lane = threadIdx.x & 31;
    const int g_begin = __ldg(a.group_begin + b), g_end = __ldg(a.group_end + b);
    if (g_begin < 0 || g_end < g_begin || g_end > a.g_max || g_end - g_begin > a.max_groups) {
        if (blockIdx.x == 0 && threadIdx.x == 0) set_error(a.err, QSA_DEVERR_VISIBLE_RANGE);
        return;
    }
    const int64_t item = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);  // (group, KV head), heads fastest
    const int64_t gi = item / a.kv_heads;
    const int h = int(item - gi * a.kv_heads);
    if (gi >= g_end - g_begin) return;
    const int64_t g = g_begin + gi;
    const int blk = __ldg(a.block_map + __ldg(a.block_offset + b) + g);
    if (blk < 0 || blk >= a.num_blocks) {
        if (lane == 0) set_error(a.err, QSA_DEVERR_SLOT_RANGE);
        return;
    }
    const int32_t *smap = a.slot_map + __ldg(a.slot_offset + b) + 4 * g;
    int64_t row[4];  // element offset of each token's row, -1 for a slot outside the cache
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int slot = __ldg(smap + u);
        const bool ok = slot >= 0 && slot < a.num_slots;
        if (!ok && lane == 0) set_error(a.err, QSA_DEVERR_SLOT_RANGE);
        row[u] = ok ? (int64_t(slot) * a.kv_heads + h) * D : -1;
    }
    uint8_t *dst = a.codes + (int64_t(blk) * a.kv_heads + h) * (8 * D);
    float *sdst = a.scales + (int64_t(blk) * a.kv_heads + h) * 2;
    auto load = [&](const float *cache, int l, float4 (&r)[4]) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
            r[u] = row[u] >= 0 ? __ldg(reinterpret_cast<const float4 *>(cache + row[u]) + l)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    if constexpr (D == 128) {  // the warp takes K, then V; both are loaded first
        float4 k[4], v[4];
        load(a.k_cache, lane, k);
        load(a.v_cache, lane, v);
        code_rows<D, kInt8>(k, lane, true, dst, sdst);
        code_rows<D, kInt8>(v, lane, false, dst, sdst + 1);
    } else {                   // lanes 0..15 take K, lanes 16..31 V
        const bool is_k = lane < 16;
        float4 r[4];
        load(is_k ? a.k_cache : a.v_cache, lane & 15, r);
        code_rows<D, kInt8>(r, lane & 15, is_k, dst, sdst + (is_k ? 0 : 1));
    }
}

}  // namespace

cudaError_t launch_code_groups(const CodeArgs &a, cudaStream_t s)
{
    if (a.batch == 0 || a.max_groups == 0) return cudaSuccess;
    const int64_t blocks = (int64_t(a.max_groups) * a.kv_heads + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    const dim3 grid(unsigned(blocks), unsigned(a.batch));
    const bool i8 = a.format == QSA_CODE_INT8;
    if (a.head_dim == 128) {
        if (i8) code_groups_kernel<128, true><<<grid, kThreads, 0, s>>>(a);
        else code_groups_kernel<128, false><<<grid, kThreads, 0, s>>>(a);
    } else if (a.head_dim == 64) {
        if (i8) code_groups_kernel<64, true><<<grid, kThreads, 0, s>>>(a);
        else code_groups_kernel<64, false><<<grid, kThreads, 0, s>>>(a);
    } else {
        return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

}  // namespace qsa
