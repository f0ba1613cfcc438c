// append.cu -- the new tokens' projected rows normalised per head, rotated and
// written where the path reads them (include/qsa_rows.h: qsa_append_tokens).
//
// Mathematics.  y = x * w * (mean(x^2) + eps)^(-1/2) per head; pairs of dims turn by
// angle_j = sum_a pos_a * freq_aj.  Far positions times binary32 frequencies lose the
// angle's fraction of a turn in binary32, so the turns are kept in 64-bit fixed point:
// F = freq / (2 pi) as a fraction of a turn, to half of 2^-64, is made once per CTA by an
// integer product with 1/(2 pi), and the axes' sum of pos * F modulo 2^64 is the angle modulo a
// full turn for every position: each F is off by 2^-65 (and the 2^-72 that its product leaves out)
// times at most 2^31, and the sum is rounded to 2^-32 once, below (axes + 3) * 2^-34 in all.  Its
// nearest quarter is taken off in integers, and sine and cosine of the rest are short Taylor series.
//
// Layout.  Partners sit in one lane: it holds eight neighbouring dims of a head's first half and
// the eight that turn with them (neighbours, or nothing turned: of its second half), so a head is a
// sixteenth of its width in lanes and half a warp takes 2, 4 or 8 heads of one projection (a step) of
// a token, the other half those of the next.  Rows come in 16-byte pieces as they lie, a batch of
// tokens ahead, through shared memory, and leave in 32-byte ones.  A warp keeps its step and walks over
// batches of tokens; the CTA's warps are a token's steps and make its table of cos and sin together.
// Visible lengths, offsets and positions come two batches ahead, slots one, none of them through a register.
//
// Bound: memory, as it does reads and twice as many writes, mostly: 32,768 tokens of 16 + 2 + 2 heads x 128
// and 8 + 1 x 64 (bf16, three axes, 616 MB): 105 us, 5.9 TB/s; without norm and rotation 109 (the same work
// in other orders of loads and stores 98-107).  Steps to that (us for 16,384 tokens): a warp per token with
// 4 dims a lane 116, a step per warp 82, loads a batch ahead through shared memory 68, eight dims a lane and
// partners by shuffles 62, partners in the lane 59, two tokens a warp and what they are looked up by without a
// register 52.  A step of 32 tokens is bound by the call (5 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache_internal.cuh"

namespace qsa {
namespace {

constexpr int kMaxWarps = 16;
constexpr int kMaxWidth = 128;
constexpr int kTokens = 8;             // of a CTA at a time, at most (32-bit rows: half as many)
constexpr int kRegisters = 72;
constexpr size_t kSmemMost = 227 * 1024;

// What a batch of tokens is looked up by, on its way through four places: two batches ahead of the arithmetic it
// is asked for, one ahead it is there.
struct Lookup {
    int64_t slot_offset[kTokens], key_offset[kTokens];
    int32_t visible[kTokens], slot[kTokens];
    int32_t position[QSA_MAX_AXES][kTokens];
};
struct Table {
    // by family: heads of d, heads of d_I.  The lower half is a signed number, and the upper one makes up for that
    uint64_t turns[2][QSA_MAX_AXES][kMaxWidth / 2];
    float norm[2][2][kMaxWidth];                     // weights of dim i at place_of(i): q, k; q_idx, idx_key
    float bad[2][kMaxWidth / 2];                     // NaN for a pair with a frequency out of range, else 0
    Lookup lookup[4];
};

// Even quads, then odd ones: a lane reads two neighbouring quads, so its reads are free of bank conflicts.
__device__ __forceinline__ int place_of(int i, int width) { return (i / 4 % 2) * (width / 2) + i / 8 * 4 + i % 4; }

// Behind the table, for the tokens of two batches: cosines and sines of d, then of d_I dims -- halves, of pair
// j at place_of(j); neighbours, of dims 2j and 2j + 1 there, the sine as the dim's partner is multiplied with it.
template <int D, int DI>
__host__ __device__ constexpr int angle_bytes() { return 2 * (D + DI) * int(sizeof(float)); }  // of a token
template <int D, int DI, int kFamily>
__device__ __forceinline__ float *angles_of(Table &table, int token)
{
    return reinterpret_cast<float *>(&table + 1) + token * (2 * (D + DI)) + (kFamily == 0 ? 0 : 2 * D);
}

// f / (2 pi) as a fraction of a turn (modulo 1, in units of 2^-64, to the nearest) for |f| < 2^16.
__device__ __forceinline__ uint64_t turns_of(float f)
{
    const uint32_t bits = __float_as_uint(f);
    const int e = int((bits >> 23) & 255u) - 127;
    if (e < -126) return 0;                      // below the smallest normal float: no turn at any position
    const uint64_t m = (bits & 0x7fffffu) | 0x800000u;
    // 1/(2 pi) = 0x28be60db9391054a7f09d5f47d4d3770 * 2^-128; f = m * 2^(e - 23)
    const unsigned __int128 lo = (unsigned __int128)m * 0x7f09d5f47d4d3770ull;
    const unsigned __int128 p = (unsigned __int128)m * 0x28be60db9391054aull + (lo >> 64);
    const int shift = 23 - e;                    // 8 .. 149
    const uint64_t t = shift < 128 ? uint64_t(((p >> (shift - 1)) + 1) >> 1) : 0;
    return bits >> 31 ? 0 - t : t;
}

// Two binary32 operations in one instruction, each rounded to nearest.
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 r;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\tfma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

// N neighbouring elements, in binary32.
template <typename T, int N>
__device__ __forceinline__ void widen(const T *p, float2 *x)
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const float4 v = reinterpret_cast<const float4 *>(p)[i];
            x[2 * i] = make_float2(v.x, v.y);
            x[2 * i + 1] = make_float2(v.z, v.w);
        }
    } else {
        uint32_t w[N / 2];
        if constexpr (N == 8) *reinterpret_cast<uint4 *>(w) = *reinterpret_cast<const uint4 *>(p);
        else *reinterpret_cast<uint2 *>(w) = *reinterpret_cast<const uint2 *>(p);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            if constexpr (std::is_same<T, __nv_bfloat16>::value)
                x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
            else
                x[i] = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        }
    }
}

__device__ __forceinline__ void store4(float *p, const float2 *x) { *reinterpret_cast<float4 *>(p) = make_float4(x[0].x, x[0].y, x[1].x, x[1].y); }
__device__ __forceinline__ void store8(float *p, const float2 *x)  // 32-byte aligned
{
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(x[0].x), "f"(x[0].y), "f"(x[1].x),
                 "f"(x[1].y), "f"(x[2].x), "f"(x[2].y), "f"(x[3].x), "f"(x[3].y)
                 : "memory");
}

// What a thread makes of a batch's angles: pair p of each u-th token.
struct Angle {
    int p, p_step, u, u_step;
};

template <int D, int DI>
__device__ __forceinline__ void make_angles(const AppendArgs &a, Table &table, const Lookup &at, const Angle &mine, int pairs0, int pairs,
                                            int token0, int n)
{
    for (int p = mine.p; p < pairs; p += mine.p_step) {
        const int fam = p < pairs0 ? 0 : 1, j = fam == 0 ? p : p - pairs0, width = fam == 0 ? D : DI;
        const bool neighbours = fam == 0 ? a.family[0].neighbours : a.family[1].neighbours;
        const int to = place_of(neighbours ? 2 * j : j, width);
        const float bad = table.bad[fam][j];
        for (int u = mine.u; u < n; u += mine.u_step) {
            uint64_t low = 1u << 31;  // the products' sum modulo 2^64, rounded to its upper half: the lower halves' part
            uint32_t phase = 0;       // .. and the upper halves'
#pragma unroll
            for (int x = 0; x < QSA_MAX_AXES; ++x)
                if (x < a.axes) {
                    const uint64_t t = table.turns[fam][x][j];
                    const int pos = at.position[x][u];
                    low += uint64_t(int64_t(pos) * int32_t(t));
                    phase += uint32_t(pos) * uint32_t(t >> 32);
                }
            phase += uint32_t(low >> 32);
            // in integers to the nearest quarter of a turn; of the rest x, at most pi/4 in size, the Taylor series
            // to x^9 and x^8 (what is left out is below 2e-9 and 3e-8)
            const uint32_t quarter = (phase + (1u << 29)) >> 30;
            const float x = float(int32_t(phase - (quarter << 30))) * 1.46291807926715968e-9f;  // 2 pi / 2^32
            const float x2 = x * x;
            float s = x2 * fmaf(x2, fmaf(x2, fmaf(x2, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6);
            float c = fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, 1.0f / 40320, -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
            s = fmaf(x, s, x);
            if (quarter & 1u) {
                const float t = c;
                c = -s;
                s = t;
            }
            if (quarter & 2u) c = -c, s = -s;
            c += bad;
            s += bad;
            float *const cosine = (fam == 0 ? angles_of<D, DI, 0>(table, token0 + u) : angles_of<D, DI, 1>(table, token0 + u)) + to;
            float *const sine = cosine + width;
            if (neighbours) {
                *reinterpret_cast<float2 *>(cosine) = make_float2(c, c);
                *reinterpret_cast<float2 *>(sine) = make_float2(-s, s);
            } else {
                *cosine = c;
                *sine = s;
            }
        }
    }
}

// All of the CTA's warps, whichever family's step each takes: they come here from different instantiations, so
// the barrier is one with a count of threads (__syncthreads() would have to be the same one for all).  It needs
// both to run the same number of rounds, which the batch, the tokens at a time and the grid alone decide.
__device__ __forceinline__ void meet_all_steps() { asm volatile("barrier.cta.sync 1, %0;" ::"r"(blockDim.x) : "memory"); }
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N, typename V>
__device__ __forceinline__ void copy_async(V *to, const V *from)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(to)), "l"(from), "n"(N) : "memory");
}

// What holds for all tokens: the norms' weights, under way when it returns, and the turns per step of each axis.
template <int D, int DI>
__device__ __forceinline__ void fetch_norms(const AppendArgs &a, Table &table)
{
    for (int i = threadIdx.x; i < 2 * (D + DI); i += blockDim.x) {
        const int fam = i < 2 * D ? 0 : 1, j = fam == 0 ? i : i - 2 * D, width = fam == 0 ? D : DI, kind = j >= width;
        const float *norm = fam == 0 ? (kind ? a.family[0].norm[1] : a.family[0].norm[0]) : (kind ? a.family[1].norm[1] : a.family[1].norm[0]);
        const int at = j - kind * width;
        if (norm != nullptr) copy_async<4>(&table.norm[fam][kind][place_of(at, kMaxWidth)], norm + at);
    }
}
__device__ __forceinline__ void make_turns(const AppendArgs &a, Table &table, int pairs0, int pairs)
{
    for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
        const int fam = i < pairs0 ? 0 : 1, j = fam == 0 ? i : i - pairs0, n = fam == 0 ? pairs0 : pairs - pairs0;
        const float *const freq = (fam == 0 ? a.family[0].freq : a.family[1].freq) + j;
        float f[QSA_MAX_AXES], bad = 0.0f;
#pragma unroll
        for (int x = 0; x < QSA_MAX_AXES; ++x) f[x] = x < a.axes ? __ldg(freq + x * n) : 0.0f;
        for (int x = 0; x < a.axes; ++x) {
            const float now = x == 0 ? f[0] : x == 1 ? f[1] : x == 2 ? f[2] : f[3];
            const bool ok = fabsf(now) < 65536.0f;
            const uint64_t t = ok ? turns_of(now) : 0;
            table.turns[fam][x][j] = t + ((t & 0x80000000u) << 1);
            if (!ok) bad = __int_as_float(0x7fffffff);
        }
        table.bad[fam][j] = bad;
    }
}

// What tokens first .. first + n - 1 are looked up by, but for their slots, into `to`.
__device__ __forceinline__ void look_up(const AppendArgs &a, Lookup &to, int first, int n)
{
    for (int i = threadIdx.x; i < (3 + QSA_MAX_AXES) * kTokens; i += blockDim.x) {
        const int what = i / kTokens, u = i % kTokens, b = first + u;
        if (u >= n) continue;
        if (what == 0) copy_async<4>(&to.visible[u], a.visible + b);
        else if (what == 1 && a.family[0].heads[1] + a.family[0].heads[2] > 0) copy_async<8>(&to.slot_offset[u], a.slot_offset + b);
        else if (what == 2 && a.family[1].heads[1] > 0) copy_async<8>(&to.key_offset[u], a.key_offset + b);
        else if (what >= 3 && what - 3 < a.axes && a.positions != nullptr)
            copy_async<4>(&to.position[what - 3][u], a.positions + int64_t(what - 3) * a.batch + b);
    }
}
// .. and, once that is there, their slots.
__device__ __forceinline__ void look_up_slots(const AppendArgs &a, Lookup &at, int n)
{
    const int u = threadIdx.x;
    if (u < n && a.family[0].heads[1] + a.family[0].heads[2] > 0) {
        const int vis = at.visible[u];
        if (vis > 0 && vis <= a.max_visible) copy_async<4>(&at.slot[u], a.slot_map + at.slot_offset[u] + vis - 1);
    }
    commit();
}

// Step `step` of one family for all the CTA's tokens, a.tokens at a time: batches blockIdx.x,
// blockIdx.x + gridDim.x, ..  Control is the same for the whole warp throughout, but for a rotation of a part of a head,
// and barriers and rounds are the same for both families.
template <typename T, int D, int DI, int kFamily>
__device__ __forceinline__ void append_step(const AppendArgs &a, Table &table, T *ring, const Angle &mine, int pairs0, int pairs, int step)
{
    constexpr int W = kFamily == 0 ? D : DI;
    constexpr int kMost = sizeof(T) == 4 ? kTokens / 2 : kTokens;
    // Turns of a warp whose instructions are mixed: two hide each other's latencies (the prompt below 105 us instead of
    // 111), but not without registers for 32-bit rows (58 instead of 51 for 12,000 tokens) or for few warps (d = 64:
    // 21 instead of 18)
    constexpr int kTogether = sizeof(T) == 2 && D == 128 ? 2 : 1;
    constexpr int kRows = 256 / W;   // heads of a step
    constexpr int kLanes = W / 16;   // lanes of a head of a token; the other half of the warp has the next token
    const int lane = threadIdx.x & 31, l = lane % kLanes;
    const AppendFamily &f = a.family[kFamily];
    const bool any = step < f.steps;
    int kind = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (kind == k && step >= f.kind_steps[k]) step -= f.kind_steps[k], kind = k + 1;
    const int heads = any ? f.heads[kind] : 0;
    const bool there = step * kRows + lane % 16 / kLanes < heads;
    // the dims are cut into pairs of quads: halves, partners, then one quad of each half of what is left (all that
    // there is for neighbours).  Pairs 2l and 2l + 1 are this lane's, eight dims at e and eight at e + apart, unless
    // the halves are cut within a lane's pairs
    const int dims = any && !(kFamily == 0 && kind == 2) ? f.dims : 0, paired = f.neighbours ? 0 : dims;
    const bool beside = paired % 16 == 0, wide = beside && f.wide;
    const int e = 16 * l < paired ? 8 * l : paired / 2 + 8 * l, apart = 16 * l < paired ? paired / 2 : (W - paired) / 2;
    auto dim_of = [&](int i) {       // of quad i: the first of both pairs, then the second ones
        const int p = 2 * l + i % 2;
        return 8 * p < paired ? 4 * p + i / 2 * (paired / 2) : paired / 2 + 4 * p + i / 2 * ((W - paired) / 2);
    };
    float *const dst = f.out[kind] + int64_t(step * kRows + lane % 16 / kLanes) * W;
    const bool normed = any && f.norm[kind] != nullptr;
    const float *const weights = table.norm[kFamily][kind & 1];

    // a batch's loads go out a batch ahead, the warp's heads of its tokens to ring[u * 8 * threads] as they
    // lie in memory: 16 bytes a lane and piece
    constexpr int kPiece = 16 / sizeof(T), kPieces = 8 / kPiece;
    const int token_bytes = 8 * int(sizeof(T)) * blockDim.x;
    ring += 8 * (threadIdx.x - lane);
    const bool mine_there = step * kRows + lane / (W / 8) < heads;
    const int64_t stride = f.stride[kind];
    const T *src = static_cast<const T *>(f.rows[kind]) + int64_t(step) * 256 + lane / (W / 8) * W + lane % (W / 8) * kPiece;
    const uint32_t ring_to = smem_u32(ring + lane / (W / 8) * W + lane % (W / 8) * kPiece);
    auto fetch = [&](int first, int buffer) {
        const int n = mine_there ? min(a.tokens, a.batch - first) : 0;
        const T *p = src + first * stride;
        uint32_t to = ring_to + buffer * (a.tokens * token_bytes);
#pragma unroll
        for (int u = 0; u < kMost; ++u, p += stride, to += token_bytes)
            if (u < n) {
#pragma unroll
                for (int i = 0; i < kPieces; ++i)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * (W / kPieces * int(sizeof(T)))), "l"(p + i * (W / kPieces)) : "memory");
            }
    };
    // Before a batch's arithmetic everything is asked for that the next one needs; its angles are made
    // behind it, into the other half, which every warp is done with since the last barrier.
    const int stepped = int(gridDim.x) * a.tokens;
    int first = int(blockIdx.x) * a.tokens, buffer = 0, turn = 0;
    auto tokens_at = [&](int first) { return min(a.tokens, a.batch - first); };
    look_up(a, table.lookup[0], first, tokens_at(first));
    look_up(a, table.lookup[1], first + stepped, tokens_at(first + stepped));
    commit();
    fetch_norms<D, DI>(a, table);
    fetch(first, 0);
    commit();
    make_turns(a, table, pairs0, pairs);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    meet_all_steps();
    look_up_slots(a, table.lookup[0], tokens_at(first));
    make_angles<D, DI>(a, table, table.lookup[0], mine, pairs0, pairs, 0, tokens_at(first));
    while (first < a.batch) {
        const int n = tokens_at(first), next = first + stepped;
        __syncwarp();  // (the lanes are done with that half)
        fetch(next, buffer ^ 1);
        look_up(a, table.lookup[(turn + 2) % 4], next + stepped, tokens_at(next + stepped));
        commit();
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        meet_all_steps();
        const Lookup &at = table.lookup[turn];
        look_up_slots(a, table.lookup[(turn + 1) % 4], tokens_at(next));
#pragma unroll kTogether
        for (int u0 = 0; u0 < n; u0 += 2) {
            const int u = u0 + lane / 16, token = buffer * a.tokens + min(u, n - 1);
            float2 x[8];             // the first quads of both pairs, then the second ones
            const T *const row = ring + token * (8 * int(blockDim.x)) + lane % 16 / kLanes * W;
            if (beside) {
                widen<T, 8>(row + e, x);
                widen<T, 8>(row + e + apart, x + 4);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) widen<T, 4>(row + dim_of(i), x + 2 * i);
            }
            if (normed) {
                auto mean_square = [&](float eps) {
                    float2 sq = mul2(x[0], x[0]);
#pragma unroll
                    for (int i = 1; i < 8; ++i) sq = fma2(x[i], x[i], sq);
                    float ss = sq.x + sq.y;
#pragma unroll
                    for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    return fmaf(ss, 1.0f / W, eps);
                };
                float mean = mean_square(a.eps);
                if (__any_sync(0xffffffffu, mean < 0x1p-100f)) {  // squares that lose bits, or all of them: of 2^96 x
                    const float up = mean < 0x1p-100f ? 0x1p96f : 1.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = mul2(x[i], make_float2(up, up));
                    mean = mean_square(a.eps * up * up);
                }
                const float r = rsqrtf(mean);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = beside ? (e + i / 2 * apart) / 2 + i % 2 * (kMaxWidth / 2) : place_of(dim_of(i), kMaxWidth);
                    const float4 w = *reinterpret_cast<const float4 *>(weights + at);
                    x[2 * i] = mul2(mul2(x[2 * i], make_float2(r, r)), make_float2(w.x, w.y));
                    x[2 * i + 1] = mul2(mul2(x[2 * i + 1], make_float2(r, r)), make_float2(w.z, w.w));
                }
            }
            const float *const cosine = angles_of<D, DI, kFamily>(table, token), *const sine = cosine + W;
            if (paired > 0) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (16 * l + 8 * h >= paired) continue;
                    const float4 c = *reinterpret_cast<const float4 *>(cosine + h * (W / 2) + 4 * l);
                    const float4 s = *reinterpret_cast<const float4 *>(sine + h * (W / 2) + 4 * l);
                    const float2 c2[2] = {make_float2(c.x, c.y), make_float2(c.z, c.w)};
                    const float2 s2[2] = {make_float2(s.x, s.y), make_float2(s.z, s.w)};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float2 &y0 = x[2 * h + i], &y1 = x[4 + 2 * h + i];
                        const float2 z = fma2(y1, c2[i], mul2(y0, s2[i])), t = mul2(y1, s2[i]);
                        y0 = make_float2(fmaf(y0.x, c2[i].x, -t.x), fmaf(y0.y, c2[i].y, -t.y));
                        y1 = z;
                    }
                }
            } else if (dims > 0) {  // neighbours
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int d = 8 * l + 4 * (i % 2) + i / 2 * (W / 2);
                    if (d >= dims) continue;
                    const float4 c = *reinterpret_cast<const float4 *>(cosine + place_of(d, W));
                    const float4 s = *reinterpret_cast<const float4 *>(sine + place_of(d, W));
                    float2 &y0 = x[2 * i], &y1 = x[2 * i + 1];
                    y0 = fma2(y0, make_float2(c.x, c.y), mul2(make_float2(y0.y, y0.x), make_float2(s.x, s.y)));
                    y1 = fma2(y1, make_float2(c.z, c.w), mul2(make_float2(y1.y, y1.x), make_float2(s.z, s.w)));
                }
            }
            if (!there || u >= n) continue;
            const int vis = at.visible[u];
            if (vis <= 0 || vis > a.max_visible) {
                if (vis != 0) {  // out of range: zero rows of its queries, and nothing else
                    set_error(a.err, QSA_DEVERR_VISIBLE_RANGE);
                    float *const p = dst + int64_t(first + u) * (heads * W) + 16 * l;
                    if (kind == 0)
#pragma unroll
                        for (int i = 0; i < 4; ++i) reinterpret_cast<float4 *>(p)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
                continue;
            }
            int64_t to;              // row of `out`
            if (kind == 0) {
                to = first + u;
            } else if (kFamily == 1) {
                to = at.key_offset[u] + vis - 1;
            } else {
                to = at.slot[u];
                if (to < 0 || to >= a.num_slots) {
                    set_error(a.err, QSA_DEVERR_SLOT_RANGE);
                    continue;
                }
            }
            float *const p = dst + to * (heads * W);
            if (wide) {
                store8(p + e, x);
                store8(p + e + apart, x + 4);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) store4(p + dim_of(i), x + 2 * i);
            }
        }
        __syncwarp();
        first = next;
        buffer ^= 1;
        turn = (turn + 1) % 4;
        make_angles<D, DI>(a, table, table.lookup[turn], mine, pairs0, pairs, buffer * a.tokens, tokens_at(first));
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// A CTA's warps are the steps blockIdx.y * warps .. of a token.
template <typename T, int D, int DI>
__global__ void __maxnreg__(kRegisters) append_kernel(const __grid_constant__ AppendArgs a)
{
    extern __shared__ __align__(16) unsigned char smem_raw[];  // the table; two batches' angles; two batches of rows
    Table &table = *reinterpret_cast<Table *>(smem_raw);
    T *const ring = reinterpret_cast<T *>(smem_raw + sizeof(Table) + 2 * a.tokens * angle_bytes<D, DI>());
    const int tid = threadIdx.x, threads = blockDim.x;
    wait_for_predecessor();
    const int pairs0 = a.family[0].dims / 2, pairs = pairs0 + a.family[1].dims / 2;
    // fewer threads than pairs: a thread has several pairs of every token; else one pair of some tokens
    Angle mine = {tid, threads, 0, 1};
    if (pairs > 0 && threads >= pairs) {
        mine = {tid % pairs, pairs, tid / pairs, threads / pairs};
        if (mine.u >= mine.u_step) mine.u = kTokens;
    }
    const int step = int(blockIdx.y) * (threads / 32) + __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (step < a.family[0].steps) append_step<T, D, DI, 0>(a, table, ring, mine, pairs0, pairs, step);
    else append_step<T, D, DI, 1>(a, table, ring, mine, pairs0, pairs, step - a.family[0].steps);
}

template <typename T, int D, int DI>
cudaError_t launch_t(AppendArgs a, int num_sms, cudaStream_t s)
{
    constexpr int kMost = sizeof(T) == 4 ? kTokens / 2 : kTokens;
    static bool attr_done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_done[dev]) {
        e = cudaFuncSetAttribute(append_kernel<T, D, DI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 int(kSmemMost));
        if (e != cudaSuccess) return e;
        attr_done[dev] = true;
    }
    const int steps = a.family[0].steps + a.family[1].steps, cuts = (steps + kMaxWarps - 1) / kMaxWarps;
    const int warps = (steps + cuts - 1) / cuts;
    // as many tokens at a time as leave room for 24 warps per SM (or what the registers do); fewer where all are
    // taken at once, but in twos, which a warp takes together
    const size_t token = 2 * (size_t(angle_bytes<D, DI>()) + size_t(warps) * 32 * 8 * sizeof(T));
    auto smem_of = [&](int tokens) { return sizeof(Table) + tokens * token; };
    const int by_registers = 65536 / (kRegisters * 32 * warps);
    auto ctas_of = [&](int tokens) {
        const int by_smem = int(size_t(228) * 1024 / (smem_of(tokens) + 1024));
        return by_registers < by_smem ? by_registers : by_smem;
    };
    const int wanted = (24 + warps - 1) / warps, enough = by_registers < wanted ? by_registers : wanted;
    int top = kMost;
    while (top > 2 && ctas_of(top) < enough) top -= 2;
    const int64_t resident = int64_t(num_sms) * ctas_of(top) / cuts, most = resident > 0 ? resident : 1;
    const int64_t share = a.batch <= most ? 1 : ((a.batch + most - 1) / most + 1) / 2 * 2;
    a.tokens = int(share > top ? top : share);
    const size_t smem = smem_of(a.tokens);
    if (smem > kSmemMost) return cudaErrorInvalidValue;
    const int64_t batches = (int64_t(a.batch) + a.tokens - 1) / a.tokens;
    return launch_kernel(append_kernel<T, D, DI>, dim3(unsigned(batches < most ? batches : most), unsigned(cuts)),
                         dim3(32 * warps), smem, s, true, a);
}

template <typename T>
cudaError_t launch_type(const AppendArgs &a, int d, int idx, int num_sms, cudaStream_t s)
{
    if (d == 128) return idx == 64 ? launch_t<T, 128, 64>(a, num_sms, s) : launch_t<T, 128, 32>(a, num_sms, s);
    return idx == 64 ? launch_t<T, 64, 64>(a, num_sms, s) : launch_t<T, 64, 32>(a, num_sms, s);
}

}  // namespace

cudaError_t launch_append(AppendArgs a, int type, int d, int idx, int num_sms, cudaStream_t s)
{
    if (a.batch == 0) return cudaSuccess;
    for (int i = 0; i < 2; ++i) {
        AppendFamily &f = a.family[i];
        const int rows = 256 / (i == 0 ? d : idx);
        f.steps = 0;
        f.wide = 1;
        for (const float *out : f.out) f.wide &= reinterpret_cast<uintptr_t>(out) % 32 == 0;
        for (int k = 0; k < 3; ++k) f.steps += f.kind_steps[k] = (f.heads[k] + rows - 1) / rows;
    }
    if ((int64_t(a.family[0].steps) + a.family[1].steps + kMaxWarps - 1) / kMaxWarps > 65535) return cudaErrorInvalidValue;
    if (type == QSA_ROWS_F32) return launch_type<float>(a, d, idx, num_sms, s);
    if (type == QSA_ROWS_BF16) return launch_type<__nv_bfloat16>(a, d, idx, num_sms, s);
    return launch_type<__half>(a, d, idx, num_sms, s);
}

}  // namespace qsa
