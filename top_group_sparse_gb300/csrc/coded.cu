// coded.cu -- complete groups' K/V rows turned into 8- or 4-bit codes with a scale
// per (group, KV head), for K and for V (include/qsa_cache.h: qsa_code_groups), and
// codes turned back into rows (include/qsa_rows.h: qsa_read_groups).
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
// x 2 heads x 128: 42 us, 6.1 TB/s; with a division per value (793 instead of
// about 350 instructions per warp, 60 % of the issue slots) it was 57 us.
//
// In 4 bits a lane's 4 x 4 values are one tile, so a tile's scale t never leaves the lane:
// t = e4m3(a / (c s)) and code = rn(x / (t s)) by the same quotients, t s being normal and
// above 2^-90 where s is above 2^-80.  A word of K is two tiles of a token, so lanes exchange
// their halves of it with their neighbours; a tile of V is 8 bytes of one lane.
// 25,063 groups x 2 heads x 128, int4: 43 us (235 MB, 35 at the copy rate), half of the issue
// slots; values one by one and all of them clamped 53, with 59 instead of 48 registers 50, each look-up
// behind the check of the one before it 47.
// Read back: 38 us; with the codes loaded where they are used 40, two groups a warp 41, 32 registers 43.
#include "codes4.cuh"

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

// Two binary32 operations in one instruction, each rounded to nearest.
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

// quotient() of two values, without the sign of a zero; minus_s: -s.
__device__ __forceinline__ float2 quotient2(float2 x, float minus_s, float r)
{
    float2 q = mul2(x, r);
    q = fma2(fma2(q, minus_s, x), r, q);
    return fma2(fma2(q, minus_s, x), r, q);
}

// Four codes + 8 of 4-bit integers, each in four bits, in the low half of a word (the rest is
// of no account): a sum with 1.5 * 2^23 + 8 rounds to the nearest integer, even on ties as 8 is,
// and holds it, + 8, in the low bits of a number whose others are 0 below bit 22.
__device__ __forceinline__ uint32_t four_int4(float a, float b, float c, float d)
{
    constexpr float kMagic = 12582912.0f + 8.0f;
    uint32_t r = __float_as_uint(__fadd_rn(d, kMagic));
    r = r * 16u + __float_as_uint(__fadd_rn(c, kMagic));
    r = r * 16u + __float_as_uint(__fadd_rn(b, kMagic));
    return r * 16u + __float_as_uint(__fadd_rn(a, kMagic));
}

// Pairs of values as e2m1 codes, the first in the low and the second in the high half of a byte;
// what is larger than the largest code becomes that.
__device__ __forceinline__ uint32_t bytes_e2m1(float2 a, float2 b, float2 c, float2 d)
{
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
    return r;
}

// An e4m3 number from its code, and the code of the number nearest to x >= 0.
__device__ __forceinline__ float from_e4m3(uint32_t code)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(code)));
    return __half2float(__ushort_as_half(uint16_t(h)));
}
__device__ __forceinline__ uint32_t to_e4m3(float x)
{
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(0.0f), "f"(x));
    return c & 0xffu;
}

// code_rows in 4 bits: this lane's dims are one tile.
template <int D, bool kInt4>
__device__ __forceinline__ void code_rows4(const float4 (&r)[4], int l, bool is_k, uint8_t *dst, float *scale_dst)
{
    constexpr float kTop = kInt4 ? 7.0f : 6.0f;
    float most = 0.0f;
#pragma unroll
    for (int u = 0; u < 4; ++u) most = max_abs3(max_abs3(most, r[u].x, r[u].y), r[u].z, r[u].w);
    uint32_t bits = __float_as_uint(most);
#pragma unroll
    for (int o = D / 8; o > 0; o >>= 1) bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, o));
    const bool finite = bits < 0x7f800000u;
    float s = __fmul_rn(__uint_as_float(bits), kInt4 ? 1.0f / 3136.0f : 1.0f / 2688.0f);
    if (s < 1.17549435e-38f) s = 0.0f;
    float2 y[4][2];  // [token][two dims]
#pragma unroll
    for (int u = 0; u < 4; ++u) y[u][0] = make_float2(r[u].x, r[u].y), y[u][1] = make_float2(r[u].z, r[u].w);
    uint32_t tile = 0;
    if (finite && s > 0.0f) {
        const float unit = __fmul_rn(kTop, s);
        const bool fast = s > 0x1p-80f;
        tile = to_e4m3(fast ? quotient<true>(most, unit, __frcp_rn(unit)) : __fdiv_rn(most, unit));
        const float ts = __fmul_rn(from_e4m3(tile), s);
        if (fast) {
            const float inv = __frcp_rn(ts);
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 x = y[u][j];
                    y[u][j] = quotient2(x, -ts, inv);
                    if constexpr (!kInt4) y[u][j] = make_float2(copysignf(y[u][j].x, x.x), copysignf(y[u][j].y, x.y));
                }
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int j = 0; j < 2; ++j) y[u][j] = make_float2(__fdiv_rn(y[u][j].x, ts), __fdiv_rn(y[u][j].y, ts));
        }
    }
    // A normal e4m3 number is at most 1/17 below what was rounded to it, so the quotients stay below
    // 7.44, or the e2m1 codes saturate; a subnormal one may be a third below, and 0 has no quotient.
    if (tile < 8) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                y[u][j] = tile == 0 ? make_float2(0.0f, 0.0f)
                                    : make_float2(fminf(fmaxf(y[u][j].x, -kTop), kTop), fminf(fmaxf(y[u][j].y, -kTop), kTop));
    }
    if (l == 0) *scale_dst = finite ? s : __int_as_float(0x7fffffff);
    if (is_k) {
        const int j = l / 16, c = l % 16 / 4, q = l % 4;  // tile q of dims 64j + 16c ..
        uint32_t word[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            uint32_t own, other;  // this tile's four codes of token u, where the word's first tile has them; the other's
            if constexpr (kInt4) own = four_int4(y[u][0].x, y[u][0].y, y[u][1].x, y[u][1].y);
            else own = bytes_e2m1(make_float2(y[u][0].x, 0.f), make_float2(y[u][0].y, 0.f), make_float2(y[u][1].x, 0.f), make_float2(y[u][1].y, 0.f));
            other = __shfl_xor_sync(D == 128 ? 0xffffffffu : 0x0000ffffu, own, 1);  // (d = 64: the lanes that take K)
            if constexpr (kInt4) word[u] = q % 2 == 0 ? __byte_perm(own, other, 0x5410) : __byte_perm(other, own, 0x5410);
            else word[u] = q % 2 == 0 ? own | other << 4 : other | own << 4;
        }
        // of the two words w = q/2 of tokens 2t + i, this lane stores those of t = q%2
        uint8_t *to = dst + j * 128 + c * 16 + (q % 2) * 8 + (q / 2) * 4;
        *reinterpret_cast<uint32_t *>(to) = q % 2 == 0 ? word[0] : word[2];
        *reinterpret_cast<uint32_t *>(to + 64) = q % 2 == 0 ? word[1] : word[3];
        dst[4 * D + c * (D / 16) + 4 * j + q] = uint8_t(tile);
    } else {
        uint32_t word[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            if constexpr (kInt4)  // tokens 0 and 2 of the word's two dims in the low half, 1 and 3 in the high one
                word[w] = __byte_perm(four_int4(y[0][w].x, y[2][w].x, y[0][w].y, y[2][w].y),
                                      four_int4(y[1][w].x, y[3][w].x, y[1][w].y, y[3][w].y), 0x5410);
            else
                word[w] = bytes_e2m1(make_float2(y[0][w].x, y[1][w].x), make_float2(y[2][w].x, y[3][w].x),
                                     make_float2(y[0][w].y, y[1][w].y), make_float2(y[2][w].y, y[3][w].y));
        }
        const int mn = l / 8, h = l % 8;  // dims 32 mn + 4h ..
        *reinterpret_cast<uint2 *>(dst + 2 * D + (mn / 2) * 128 + h * 16 + (mn % 2) * 8) = make_uint2(word[0], word[1]);
        dst[4 * D + D / 4 + h * (D / 32) + mn] = uint8_t(tile);
    }
}

template <int D, int kFormat>
__device__ __forceinline__ void code_rows_as(const float4 (&r)[4], int l, bool is_k, uint8_t *dst, float *scale_dst)
{
    if constexpr (is_4bit(kFormat)) code_rows4<D, kFormat == QSA_CODE_INT4>(r, l, is_k, dst, scale_dst);
    else code_rows<D, kFormat == QSA_CODE_INT8>(r, l, is_k, dst, scale_dst);
}

template <int D, int kFormat>
__global__ void __launch_bounds__(kThreads, is_4bit(kFormat) && D == 128 ? 5 : 0) code_groups_kernel(const CodeArgs a)
{
    const int b = blockIdx.y;
    const int lane = threadIdx.x & 31;
    wait_for_predecessor();
    const int g_begin = __ldg(a.group_begin + b), g_end = __ldg(a.group_end + b);
    const int64_t block_offset = __ldg(a.block_offset + b), slot_offset = __ldg(a.slot_offset + b);
    if (g_begin < 0 || g_end < g_begin || g_end > a.g_max || g_end - g_begin > a.max_groups) {
        if (blockIdx.x == 0 && threadIdx.x == 0) set_error(a.err, QSA_DEVERR_VISIBLE_RANGE);
        return;
    }
    const int64_t item = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);  // (group, KV head), heads fastest
    const int64_t gi = item / a.kv_heads;
    const int h = int(item - gi * a.kv_heads);
    if (gi >= g_end - g_begin) return;
    const int64_t g = g_begin + gi;
    const int blk = __ldg(a.block_map + block_offset + g);
    const int32_t *smap = a.slot_map + slot_offset + 4 * g;
    int64_t row[4];  // element offset of each token's row, -1 for a slot outside the cache
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int slot = __ldg(smap + u);
        const bool ok = slot >= 0 && slot < a.num_slots;
        if (!ok && lane == 0) set_error(a.err, QSA_DEVERR_SLOT_RANGE);
        row[u] = ok ? (int64_t(slot) * a.kv_heads + h) * D : -1;
    }
    if (blk < 0 || blk >= a.num_blocks) {
        if (lane == 0) set_error(a.err, QSA_DEVERR_SLOT_RANGE);
        return;
    }
    uint8_t *dst = a.codes + (int64_t(blk) * a.kv_heads + h) * code_bytes(kFormat, D);
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
        code_rows_as<D, kFormat>(k, lane, true, dst, sdst);
        code_rows_as<D, kFormat>(v, lane, false, dst, sdst + 1);
    } else {                   // lanes 0..15 take K, lanes 16..31 V
        const bool is_k = lane < 16;
        float4 r[4];
        load(is_k ? a.k_cache : a.v_cache, lane & 15, r);
        code_rows_as<D, kFormat>(r, lane & 15, is_k, dst, sdst + (is_k ? 0 : 1));
    }
}

// ---- the way back ---------------------------------------------------------------------
// Values of this lane's dims (4*l .. 4*l+3) of the four tokens of a (group, head), K or V.
// A product of a code and its tile's scale is exact in binary32.

// What a lane loads for them.
struct Loaded {
    uint32_t w[4], tile;
    float s;
};

template <int D, int F>
__device__ __forceinline__ Loaded load_codes(const uint8_t *src, const float *scales, int l, bool is_k)
{
    Loaded x{};
    x.s = __ldg(scales + (is_k ? 0 : 1));
    if constexpr (is_4bit(F)) {
        const int j = l / 16, c = l % 16 / 4, q = l % 4, mn = l / 8, h = l % 8;
        x.tile = __ldg(src + 4 * D + (is_k ? c * (D / 16) + 4 * j + q : D / 4 + h * (D / 32) + mn));
        if (is_k) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                x.w[u] = __ldg(reinterpret_cast<const uint32_t *>(src + j * 128 + (u % 2) * 64 + c * 16 + (u / 2) * 8 + (q / 2) * 4));
        } else {
            const uint2 v = __ldg(reinterpret_cast<const uint2 *>(src + 2 * D + (mn / 2) * 128 + h * 16 + (mn % 2) * 8));
            x.w[0] = v.x, x.w[1] = v.y;
        }
    } else if (is_k) {
#pragma unroll
        for (int u = 0; u < 4; ++u) x.w[u] = __ldg(reinterpret_cast<const uint32_t *>(src + (l / 16) * 256 + u * 64 + (l % 16) * 4));
    } else {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src + 4 * D + l * 16));
        x.w[0] = v.x, x.w[1] = v.y, x.w[2] = v.z, x.w[3] = v.w;
    }
    return x;
}

// The number that byte u of a word of 8-bit codes stands for.
template <bool kInt8>
__device__ __forceinline__ float from_byte(uint32_t word, int u)
{
    return kInt8 ? float(int8_t(word >> (8 * u))) : from_e4m3(word >> (8 * u) & 0xffu);
}

template <int F>
__device__ __forceinline__ void values_of(const Loaded &x, int l, bool is_k, const Int4Base &base, float4 (&r)[4])
{
    if constexpr (is_4bit(F)) {
        const TileScale<F> ts(two_e4m3(x.tile * 0x101u));
        auto value = [&](uint32_t two) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&two));
            return mul2(F == QSA_CODE_INT4 ? mul2(v, kUnits<F>) : v, x.s);
        };
        if (is_k) {
            const int q = l % 4;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                // this tile's half of the word, its codes brought to where decode_word has the pairs 0 and 2
                uint32_t own, d[4];
                if constexpr (F == QSA_CODE_INT4) {
                    own = q % 2 == 0 ? x.w[u] : x.w[u] >> 16;
                    own = (own & 0x0f0fu) | (own & 0xf0f0u) << 12;
                } else {
                    own = (q % 2 == 0 ? x.w[u] : x.w[u] >> 4) & 0x0f0f0f0fu;
                    own |= own >> 4;
                }
                decode_word<F>(own, ts, base, d);
                const float2 a = value(d[0]), b = value(d[2]);
                r[u] = make_float4(a.x, a.y, b.x, b.y);
            }
        } else {
            uint32_t d[2][4];
            decode_word<F>(x.w[0], ts, base, d[0]);
            decode_word<F>(x.w[1], ts, base, d[1]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {  // tokens 2u and 2u + 1
                const float2 y0 = value(d[0][u]), y1 = value(d[0][2 + u]), y2 = value(d[1][u]), y3 = value(d[1][2 + u]);
                r[2 * u] = make_float4(y0.x, y1.x, y2.x, y3.x);
                r[2 * u + 1] = make_float4(y0.y, y1.y, y2.y, y3.y);
            }
        }
    } else {
        constexpr bool kInt8 = F == QSA_CODE_INT8;
#pragma unroll
        for (int u = 0; u < 4; ++u) {  // K: of token u's word, V: byte u of a dim's
            if (is_k)
                r[u] = make_float4(from_byte<kInt8>(x.w[u], 0) * x.s, from_byte<kInt8>(x.w[u], 1) * x.s,
                                   from_byte<kInt8>(x.w[u], 2) * x.s, from_byte<kInt8>(x.w[u], 3) * x.s);
            else
                r[u] = make_float4(from_byte<kInt8>(x.w[0], u) * x.s, from_byte<kInt8>(x.w[1], u) * x.s,
                                   from_byte<kInt8>(x.w[2], u) * x.s, from_byte<kInt8>(x.w[3], u) * x.s);
        }
    }
}

// Bound by memory, by its stores: a warp takes one (group, head), asks for all of its codes at
// once, and writes 32*d bytes of rows in whole 16-byte pieces.
template <int D, int kFormat>
__global__ void __launch_bounds__(kThreads, 6) read_groups_kernel(const CodeArgs a)
{
    const int b = blockIdx.y;
    const int lane = threadIdx.x & 31;
    wait_for_predecessor();
    const int g_begin = __ldg(a.group_begin + b), g_end = __ldg(a.group_end + b);
    const int64_t block_offset = __ldg(a.block_offset + b), slot_offset = __ldg(a.slot_offset + b);
    if (g_begin < 0 || g_end < g_begin || g_end > a.g_max || g_end - g_begin > a.max_groups) {
        if (blockIdx.x == 0 && threadIdx.x == 0) set_error(a.err, QSA_DEVERR_VISIBLE_RANGE);
        return;
    }
    const int64_t item = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);  // (group, KV head), heads fastest
    const int64_t gi = item / a.kv_heads;
    const int h = int(item - gi * a.kv_heads);
    if (gi >= g_end - g_begin) return;
    const int64_t g = g_begin + gi;
    const int blk = __ldg(a.block_map + block_offset + g);
    int slot[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) slot[u] = __ldg(a.slot_map + slot_offset + 4 * g + u);
    const bool there = blk >= 0 && blk < a.num_blocks;
    constexpr int kSides = D == 128 ? 2 : 1;  // K and V, or the one that this half of the warp takes
    const int l = D == 128 ? lane : lane & 15;
    Loaded x[kSides];
#pragma unroll
    for (int k = 0; k < kSides; ++k) {
        x[k] = Loaded{};
        const int64_t at = int64_t(blk) * a.kv_heads + h;
        if (there) x[k] = load_codes<D, kFormat>(a.codes + at * code_bytes(kFormat, D), a.scales + 2 * at, l, kSides == 2 ? k == 0 : lane < 16);
    }
    if (!there && lane == 0) set_error(a.err, QSA_DEVERR_SLOT_RANGE);
#pragma unroll
    for (int k = 0; k < kSides; ++k) {
        const bool is_k = kSides == 2 ? k == 0 : lane < 16;
        float4 r[4];
        values_of<kFormat>(x[k], l, is_k, Int4Base(uint32_t(a.batch >> 31)), r);
        float *cache = const_cast<float *>(is_k ? a.k_cache : a.v_cache);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (slot[u] >= 0 && slot[u] < a.num_slots)
                *(reinterpret_cast<float4 *>(cache + (int64_t(slot[u]) * a.kv_heads + h) * D) + l) =
                    there ? r[u] : make_float4(0.f, 0.f, 0.f, 0.f);
            else if (lane == 0) set_error(a.err, QSA_DEVERR_SLOT_RANGE);
        }
    }
}

template <int D>
cudaError_t launch_d(const CodeArgs &a, bool back, cudaStream_t s)
{
    const int64_t blocks = (int64_t(a.max_groups) * a.kv_heads + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    const dim3 grid(unsigned(blocks), unsigned(a.batch));
    auto launch = [&](void (*code)(const CodeArgs), void (*read)(const CodeArgs)) {
        return launch_kernel(back ? read : code, grid, dim3(kThreads), 0, s, true, a);
    };
    switch (a.format) {
        case QSA_CODE_E4M3: return launch(code_groups_kernel<D, QSA_CODE_E4M3>, read_groups_kernel<D, QSA_CODE_E4M3>);
        case QSA_CODE_INT8: return launch(code_groups_kernel<D, QSA_CODE_INT8>, read_groups_kernel<D, QSA_CODE_INT8>);
        case QSA_CODE_E2M1: return launch(code_groups_kernel<D, QSA_CODE_E2M1>, read_groups_kernel<D, QSA_CODE_E2M1>);
        case QSA_CODE_INT4: return launch(code_groups_kernel<D, QSA_CODE_INT4>, read_groups_kernel<D, QSA_CODE_INT4>);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch(const CodeArgs &a, bool back, cudaStream_t s)
{
    if (a.batch == 0 || a.max_groups == 0) return cudaSuccess;
    if (a.head_dim == 128) return launch_d<128>(a, back, s);
    if (a.head_dim == 64) return launch_d<64>(a, back, s);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_code_groups(const CodeArgs &a, cudaStream_t s) { return launch(a, false, s); }
cudaError_t launch_read_groups(const CodeArgs &a, cudaStream_t s) { return launch(a, true, s); }

}  // namespace qsa
