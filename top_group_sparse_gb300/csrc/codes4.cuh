// codes4.cuh -- 4-bit codes and their tile scales as 16-bit floats (include/qsa_cache.h: the layout).
#pragma once

#include <cuda_fp16.h>

#include "cache_internal.cuh"

namespace qsa {
namespace {

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t two_e4m3(uint32_t codes)  // the low two bytes as 16-bit floats
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(codes)));
    return r;
}

// A pair of tile scales as the decoding of 4-bit codes uses it.
template <int F>
struct TileScale {
    uint32_t t, zero, zero16;
    // int4: an eighth of the scale, so that the products with 1032 and 72 stay below 2^16; kUnits makes
    // up for it (not in the group's scale, which may be any finite number)
    __device__ __forceinline__ explicit TileScale(uint32_t pair)
    {
        if constexpr (F == QSA_CODE_INT4) {
            t = mul_f16x2(pair, 0x30003000u);       // 1/8
            zero = mul_f16x2(pair, 0xd808d808u);    // -129 = -1032 / 8
            zero16 = mul_f16x2(pair, 0xc880c880u);  // -9 = -72 / 8
        } else {
            t = pair;
        }
    }
};

// What a decoded value has to be multiplied by.
template <int F>
constexpr int kLog2Units = F == QSA_CODE_INT4 ? 3 : 0;
template <int F>
constexpr float kUnits = float(1 << kLog2Units<F>);

// What int4 codes are put into: 1024 and 64 as pairs of 16-bit floats.  A masking into a register
// is one instruction, into a second constant two (8 histories of 262,144 tokens 164 us instead of 150), so the
// compiler is not to know the values: `zero` is 0 and comes from a kernel's argument.
struct Int4Base {
    uint32_t k1024, k64;
    __device__ __forceinline__ explicit Int4Base(uint32_t zero) : k1024(0x64006400u + zero), k64(0x54005400u + zero) {}
};

// The four pairs of a word of 4-bit codes, times their tiles' scales, as pairs of 16-bit
// floats in units of kUnits.  All exact: a code has at most 3 significant bits and a scale 4.
template <int F>
__device__ __forceinline__ void decode_word(uint32_t w, const TileScale<F> &s, const Int4Base &base, uint32_t (&r)[4])
{
    if constexpr (F == QSA_CODE_INT4) {
        // code + 8 in the low bits of 1024, or four bits up in 64, is 1024 + 8 + code or 64 + 8 + code
        const uint32_t v = w >> 8;
        r[0] = fma_f16x2((w & 0x000f000fu) | base.k1024, s.t, s.zero);
        r[1] = fma_f16x2((w & 0x00f000f0u) | base.k64, s.t, s.zero16);
        r[2] = fma_f16x2((v & 0x000f000fu) | base.k1024, s.t, s.zero);
        r[3] = fma_f16x2((v & 0x00f000f0u) | base.k64, s.t, s.zero16);
    } else {
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
            : "r"(w));
#pragma unroll
        for (int p = 0; p < 4; ++p) r[p] = mul_f16x2(r[p], s.t);
    }
}

}  // namespace
}  // namespace qsa
