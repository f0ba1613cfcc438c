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
// leave from one lane, and every load is a 16-byte piece of a row.  25,063 groups
// x 2 heads x 128: 43 us, 5.9 TB/s; with a division per value (793 instead of
// about 350 instructions per warp, 60 % of the issue slots) it was 57 us.
#include "cache_internal.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// The largest of |a|, |b| and |c|; NaN if one of them is.
__device__ __forceinline__ float max_abs3(float a, float b, float c)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
    return r;
}

// x / s rounded to nearest, given r = 1/s rounded to nearest.  The first two steps
// bring q within one unit in the last place of the quotient; then, by Markstein's
// theorem (P. Markstein, Computation of elementary functions on the IBM RISC
// System/6000, 1990), one more correction by the exact remainder rounds as the
// division does.  A remainder is exact while it does not underflow: the caller
// divides where the scale is below 2^-90 (and a quotient so small that its own
// remainder underflows is far below half the smallest code).  Of x = -0 the corrections
// make +0; an e4m3 code holds the sign, so there it is x's, as a division's is.
template <bool kInt8>
__device__ __forceinline__ float quotient(float x, float s, float r)
{
    float q = __fmul_rn(x, r);
    q = __fmaf_rn(__fmaf_rn(-q, s, x), r, q);
    q = __fmaf_rn(__fmaf_rn(-q, s, x), r, q);
    return kInt8 ? q : copysignf(q, x);
}

// Four quotients of at most the format's largest code in size, as codes.
template <bool kInt8>
__device__ __forceinline__ uint32_t code4(float x, float y, float z, float w)
{
    if constexpr (kInt8) {
        // x + 1.5 * 2^23 rounds x to the nearest integer, even on ties, and holds it in its low bits
        constexpr float kMagic = 12582912.0f;
        const uint32_t lo = __byte_perm(__float_as_uint(__fadd_rn(x, kMagic)), __float_as_uint(__fadd_rn(y, kMagic)), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(__fadd_rn(z, kMagic)), __float_as_uint(__fadd_rn(w, kMagic)), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    } else {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y), "f"(x));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(w), "f"(z));
        return uint32_t(lo) | (uint32_t(hi) << 16);
    }
}

// Codes the four tokens' rows of K or V of one (group, head), D/4 lanes of 4
// dims each: r[u] are this lane's dims (4*l .. 4*l+3) of token u.  Every lane of
// the warp calls it (two halves may code different rows).
template <int D, bool kInt8>
__device__ __forceinline__ void code_rows(const float4 (&r)[4], int l, bool is_k, uint8_t *dst, float *scale_dst)
{
    float top = 0.0f;
#pragma unroll
    for (int u = 0; u < 4; ++u) top = max_abs3(max_abs3(top, r[u].x, r[u].y), r[u].z, r[u].w);
    uint32_t bits = __float_as_uint(top);  // (a NaN's are above infinity's, infinity's above every number's)
#pragma unroll
    for (int o = D / 8; o > 0; o >>= 1) bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, o));
    const bool finite = bits < 0x7f800000u;
    float s = __fmul_rn(__uint_as_float(bits), kInt8 ? 1.0f / 127.0f : 1.0f / 448.0f);
    if (s < 1.17549435e-38f) s = 0.0f;  // below the smallest normal float: flushed
    uint32_t c[4] = {0u, 0u, 0u, 0u};
    if (finite && s > 0x1p-90f) {
        const float inv = __frcp_rn(s);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            c[u] = code4<kInt8>(quotient<kInt8>(r[u].x, s, inv), quotient<kInt8>(r[u].y, s, inv),
                                quotient<kInt8>(r[u].z, s, inv), quotient<kInt8>(r[u].w, s, inv));
    } else if (finite && s > 0.0f) {
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
    wait_for_predecessor();
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
    auto launch = [&](void (*kernel)(const CodeArgs)) { return launch_kernel(kernel, grid, dim3(kThreads), 0, s, true, a); };
    if (a.head_dim == 128) return launch(i8 ? code_groups_kernel<128, true> : code_groups_kernel<128, false>);
    if (a.head_dim == 64) return launch(i8 ? code_groups_kernel<64, true> : code_groups_kernel<64, false>);
    return cudaErrorInvalidValue;
}

}  // namespace qsa
