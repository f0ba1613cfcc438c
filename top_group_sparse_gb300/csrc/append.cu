// append.cu -- the new tokens' projected rows normalised per head, rotated and
// written where the path reads them (include/qsa_rows.h: qsa_append_tokens).
//
// Mathematics.  y = x * w * (mean(x^2) + eps)^(-1/2) per head; pairs of dims turn by
// angle_j = sum_a pos_a * freq_aj.  Far positions times binary32 frequencies lose the
// angle's fraction of a turn in binary32, so the turns are kept in 64-bit fixed point:
// F = freq / (2 pi) as a fraction of a turn, exact to 2^-64, is made once per CTA by an
// integer product with 1/(2 pi), and pos * F modulo 2^64 is the angle modulo a full turn
// for every position.  Sine and cosine are then of a binary32 number of half turns.
//
// Layout.  A lane holds eight neighbouring dims (two quads), so a head is an eighth of its
// width in lanes, a warp takes 2, 4 or 8 heads of one projection (a step), and 16-bit rows
// come in 16-byte pieces and leave in 32-byte ones.  A warp keeps its step -- pointers, norm
// weights -- and walks over tokens, a few at a time whose loads are out together; the CTA's
// warps are a token's steps and make its table of cos and signed sin per dim together.  The
// partner of a dim is in the same lane (neighbours) or a fixed number of quads away (halves:
// dims is a multiple of 8), so a rotation is z = y * cos + partner * (+-sin) for both.
//
// Bound: memory, and the instructions of the norm and the rotation, by about the same.  32,768
// tokens of 16 + 2 + 2 heads x 128 and 8 + 1 x 64 (bf16, three axes, 616 MB): 124 us, 5.0 TB/s;
// without norm and rotation the same kernel streams at 6.5.  Steps to that (us for 16,384
// tokens): a warp per token with 4 dims a lane and one head ahead 116, four heads ahead 116,
// projections one after the other instead of chosen for each head 78, a step per warp as now 82,
// control the same for the whole warp 72, loads a batch ahead through shared memory 68, packed
// arithmetic and pointers kept 66.  A step of 32 tokens is bound by the call (4.9 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache_internal.cuh"

namespace qsa {
namespace {

constexpr int kMaxWarps = 16;
constexpr int kMaxWidth = 128;
constexpr int kTokens = 4;             // of a CTA at a time, at most (32-bit rows: half as many)
constexpr int kRegisters = 48;

struct Table {
    uint64_t turns[2][QSA_MAX_AXES][kMaxWidth / 2];  // by family: heads of d, heads of d_I
    float bad[2][kMaxWidth / 2];                     // NaN for a pair with a frequency out of range, else 0
    // [two batches of tokens]: of dim 8l + 4h + i at [h * width/2 + 4l + i], free of bank conflicts
    float cosine[2][kTokens][2][kMaxWidth], sine[2][kTokens][2][kMaxWidth];
};

__device__ __forceinline__ int place_of(int dim, int width) { return (dim / 4 % 2) * (width / 2) + dim / 8 * 4 + dim % 4; }

// f / (2 pi) as a fraction of a turn (modulo 1, in units of 2^-64) for |f| < 2^16.
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
    const uint64_t t = shift < 128 ? uint64_t(p >> shift) : 0;
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

// Eight elements of a row, a lane's own, on their way through shared memory.
template <typename T>
struct Raw {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void fetch(const T *p)
    {
#pragma unroll
        for (int i = 0; i < int(sizeof(T) / 2); ++i)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(v + i)), "l"(p + i * (16 / sizeof(T))) : "memory");
    }
    __device__ __forceinline__ void widen(float2 (&x)[4]) const
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[2 * i] = make_float2(__uint_as_float(v[i].x), __uint_as_float(v[i].y));
                x[2 * i + 1] = make_float2(__uint_as_float(v[i].z), __uint_as_float(v[i].w));
            }
        } else {
            const uint4 r = v[0];
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (std::is_same<T, __nv_bfloat16>::value)
                    x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
                else
                    x[i] = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            }
        }
    }
};

// 32 bytes at once where they are so aligned: in 16-byte pieces a warp's store would touch every
// 32-byte sector twice.
__device__ __forceinline__ void store(float *p, const float2 (&x)[4], bool wide)
{
    if (wide) {
        asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(x[0].x), "f"(x[0].y), "f"(x[1].x),
                     "f"(x[1].y), "f"(x[2].x), "f"(x[2].y), "f"(x[3].x), "f"(x[3].y)
                     : "memory");
    } else {
        reinterpret_cast<float4 *>(p)[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
        reinterpret_cast<float4 *>(p)[1] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
    }
}

// What a thread makes of a token's table: pair p of each u-th of a batch's tokens.
struct Angle {
    int p, p_step, u, u_step;
};
struct Position {
    int at[QSA_MAX_AXES];
};
__device__ __forceinline__ Position position_of(const AppendArgs &a, int b)
{
    Position r;
#pragma unroll
    for (int x = 0; x < QSA_MAX_AXES; ++x)
        r.at[x] = a.positions != nullptr && x < a.axes && b < a.batch ? __ldg(a.positions + int64_t(x) * a.batch + b) : 0;
    return r;
}

// `first`: the position of the first of the thread's tokens.
__device__ __forceinline__ void make_angles(const AppendArgs &a, Table &table, const Angle &mine, int pairs0, int pairs, int d, int di,
                                            int buffer, int b0, int n, const Position &first)
{
    for (int p = mine.p; p < pairs; p += mine.p_step) {
        const int fam = p < pairs0 ? 0 : 1, j = fam == 0 ? p : p - pairs0, side = fam == 0 ? pairs0 : pairs - pairs0;
        const int width = fam == 0 ? d : di;
        const bool neighbours = fam == 0 ? a.family[0].neighbours : a.family[1].neighbours;
        const int one = place_of(neighbours ? 2 * j : j, width), two = place_of(neighbours ? 2 * j + 1 : j + side, width);
        const float bad = table.bad[fam][j];
        for (int u = mine.u; u < n; u += mine.u_step) {
            const Position pos = u == mine.u ? first : position_of(a, b0 + u);
            uint32_t phase = 0;  // the upper half of the products' sum modulo 2^64, but for the lower halves' carries
#pragma unroll
            for (int x = 0; x < QSA_MAX_AXES; ++x)
                if (x < a.axes) {
                    const uint64_t t = table.turns[fam][x][j];
                    const uint32_t at = uint32_t(pos.at[x]);
                    phase += __umulhi(at, uint32_t(t)) + at * uint32_t(t >> 32) - (pos.at[x] < 0 ? uint32_t(t) : 0u);
                }
            // in integers to the nearest quarter of a turn: the rest, at most an eighth, loses a quarter as
            // much to binary32 as an angle of half a turn would
            const uint32_t quarter = (phase + (1u << 29)) >> 30;
            float s, c;
            sincospif(float(int32_t(phase - (quarter << 30))) * 0x1p-31f, &s, &c);  // half turns
            if (quarter & 1u) {
                const float t = c;
                c = -s;
                s = t;
            }
            if (quarter & 2u) c = -c, s = -s;
            float *const cosine = table.cosine[buffer][u][fam], *const sine = table.sine[buffer][u][fam];
            cosine[one] = cosine[two] = c + bad;
            sine[one] = -s + bad;
            sine[two] = s + bad;
        }
    }
}

// Step `step` of one family for all the CTA's tokens, a.tokens at a time: batches blockIdx.x,
// blockIdx.x + gridDim.x, ..  Control is the same for the whole warp throughout.
template <typename T, int W, int kFamily>
__device__ __forceinline__ void append_step(const AppendArgs &a, Table &table, Raw<T> *ring, const Angle &mine, int pairs0, int pairs, int d, int di,
                                            int step)
{
    constexpr int kMost = sizeof(T) == 4 ? kTokens / 2 : kTokens;
    constexpr int kLanes = W / 8, kRows = 32 / kLanes;
    const int lane = threadIdx.x & 31, l = lane % kLanes;
    const AppendFamily &f = a.family[kFamily];
    const bool any = step < f.steps;
    int kind = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (kind == k && step >= f.kind_steps[k]) step -= f.kind_steps[k], kind = k + 1;
    const int head = step * kRows + lane / kLanes, heads = any ? f.heads[kind] : 0;
    const bool there = head < heads;
    const T *src = static_cast<const T *>(f.rows[kind]) + int64_t(head) * W + 8 * l;
    const int64_t stride = f.stride[kind];
    float *const dst = f.out[kind] + int64_t(head) * W + 8 * l;
    const bool normed = any && f.norm[kind] != nullptr;
    float2 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = normed ? __ldg(reinterpret_cast<const float2 *>(f.norm[kind] + 8 * l) + i) : make_float2(0.f, 0.f);
    const int apart = any && !(kFamily == 0 && kind == 2) ? f.dims / 8 : 0;  // quads
    int partner[2];                  // lanes of the partners of this lane's quads (halves)
    bool turned[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int quad = 2 * l + h;
        turned[h] = quad < 2 * apart;
        partner[h] = turned[h] ? lane - l + (quad < apart ? quad + apart : quad - apart) / 2 : lane;
    }

    // a batch's loads, this lane's pieces of its tokens at ring[u * threads], go out a batch ahead
    ring += threadIdx.x;
    const int threads = blockDim.x;
    auto fetch = [&](int first, int buffer) {
        const int n = there ? min(a.tokens, a.batch - first) : 0;
        const T *p = src + first * stride;
        Raw<T> *to = ring + buffer * (kMost * threads);
#pragma unroll
        for (int u = 0; u < kMost; ++u, p += stride, to += threads)
            if (u < n) to->fetch(p);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // the elements of `out` before the row that token first + u goes to: lane u looks it up.  -1: none,
    // and of a query that is out of range -2 - that, for zeros
    auto look_up = [&](int first) {
        int64_t at = -1;
        if (lane < min(a.tokens, a.batch - first) && any) {
            const int b = first + lane, vis = __ldg(a.visible + b);
            if (vis < 0 || vis > a.max_visible) {
                set_error(a.err, QSA_DEVERR_VISIBLE_RANGE);
                at = kind == 0 ? -2 - int64_t(b) * (heads * W) : -1;
            } else if (vis > 0) {
                if (kind == 0) {
                    at = b;
                } else if (kFamily == 1) {
                    at = __ldg(a.key_offset + b) + vis - 1;
                } else {
                    const int slot = __ldg(a.slot_map + __ldg(a.slot_offset + b) + vis - 1);
                    if (slot >= 0 && slot < a.num_slots) at = slot;
                    else set_error(a.err, QSA_DEVERR_SLOT_RANGE);
                }
                if (at >= 0) at *= heads * W;
            }
        }
        return at;
    };
    // Before a batch's arithmetic everything is asked for that the next one needs; its table is made
    // behind it, into the other half, which every warp is done with since the last barrier.
    const int stepped = int(gridDim.x) * a.tokens;
    int first = int(blockIdx.x) * a.tokens, buffer = 0;
    fetch(first, 0);
    int64_t to = look_up(first);
    make_angles(a, table, mine, pairs0, pairs, d, di, 0, first, min(a.tokens, a.batch - first), position_of(a, first + mine.u));
    while (first < a.batch) {
        const int n = min(a.tokens, a.batch - first), next = first + stepped;
        fetch(next, buffer ^ 1);
        const int64_t next_to = look_up(next);
        const Position next_position = position_of(a, next + mine.u);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kMost; ++u) {
            if (u >= n) break;
            float2 x[4];
            ring[(buffer * kMost + u) * threads].widen(x);
            if (normed) {
                float2 sq = mul2(x[0], x[0]);
#pragma unroll
                for (int i = 1; i < 4; ++i) sq = fma2(x[i], x[i], sq);
                float ss = sq.x + sq.y;
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float r = rsqrtf(fmaf(ss, 1.0f / W, a.eps));
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = mul2(mul2(x[i], make_float2(r, r)), w[i]);
            }
            if (apart > 0) {
                float2 y[4];
                if (f.neighbours) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = make_float2(x[i].y, x[i].x);
                } else {
                    const bool other = apart % 2 != 0;  // an odd number of quads away: the other quad of that lane
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        y[i].x = __shfl_sync(0xffffffffu, other ? x[i ^ 2].x : x[i].x, partner[i / 2]);
                        y[i].y = __shfl_sync(0xffffffffu, other ? x[i ^ 2].y : x[i].y, partner[i / 2]);
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float4 c = *reinterpret_cast<const float4 *>(&table.cosine[buffer][u][kFamily][h * (W / 2) + 4 * l]);
                    const float4 s = *reinterpret_cast<const float4 *>(&table.sine[buffer][u][kFamily][h * (W / 2) + 4 * l]);
                    const float2 z0 = fma2(x[2 * h], make_float2(c.x, c.y), mul2(y[2 * h], make_float2(s.x, s.y)));
                    const float2 z1 = fma2(x[2 * h + 1], make_float2(c.z, c.w), mul2(y[2 * h + 1], make_float2(s.z, s.w)));
                    if (turned[h]) x[2 * h] = z0, x[2 * h + 1] = z1;
                }
            }
            int64_t at = __shfl_sync(0xffffffffu, to, u);
            if (at < -1) {
                at = -2 - at;
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = make_float2(0.0f, 0.0f);
            }
            if (there && at >= 0) store(dst + at, x, f.wide);
        }
        first = next;
        to = next_to;
        buffer ^= 1;
        make_angles(a, table, mine, pairs0, pairs, d, di, buffer, first, min(a.tokens, a.batch - first), next_position);
    }
}

// A CTA's warps are the steps blockIdx.y * warps .. of a token.
template <typename T, int D, int DI>
__global__ void __maxnreg__(kRegisters) append_kernel(const __grid_constant__ AppendArgs a)
{
    extern __shared__ __align__(16) unsigned char smem_raw[];  // the table; two batches of raw pieces
    Table &table = *reinterpret_cast<Table *>(smem_raw);
    Raw<T> *const ring = reinterpret_cast<Raw<T> *>(smem_raw + sizeof(Table));
    const int tid = threadIdx.x, threads = blockDim.x;
    wait_for_predecessor();
    const int pairs0 = a.family[0].dims / 2, pairs = pairs0 + a.family[1].dims / 2;
    for (int i = tid; i < pairs; i += threads) {
        const int fam = i < pairs0 ? 0 : 1, j = fam == 0 ? i : i - pairs0, n = fam == 0 ? pairs0 : pairs - pairs0;
        float bad = 0.0f;
        for (int x = 0; x < a.axes; ++x) {
            const float freq = __ldg((fam == 0 ? a.family[0].freq : a.family[1].freq) + x * n + j);
            const bool ok = fabsf(freq) < 65536.0f;
            table.turns[fam][x][j] = ok ? turns_of(freq) : 0;
            if (!ok) bad = __int_as_float(0x7fffffff);
        }
        table.bad[fam][j] = bad;
    }
    // fewer threads than pairs: a thread has several pairs of every token; else one pair of some tokens
    Angle mine = {tid, threads, 0, 1};
    if (pairs > 0 && threads >= pairs) {
        mine = {tid % pairs, pairs, tid / pairs, threads / pairs};
        if (mine.u >= mine.u_step) mine.u = kTokens;
    }
    __syncthreads();
    const int step = int(blockIdx.y) * (threads / 32) + __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (step < a.family[0].steps) append_step<T, D, 0>(a, table, ring, mine, pairs0, pairs, D, DI, step);
    else append_step<T, DI, 1>(a, table, ring, mine, pairs0, pairs, D, DI, step - a.family[0].steps);
}

template <typename T, int D, int DI>
cudaError_t launch_t(AppendArgs a, int num_sms, cudaStream_t s)
{
    constexpr int kMost = sizeof(T) == 4 ? kTokens / 2 : kTokens;
    constexpr size_t kRing = size_t(2) * kMost * 32 * sizeof(Raw<T>);  // of a warp
    static bool attr_done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_done[dev]) {
        e = cudaFuncSetAttribute(append_kernel<T, D, DI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 int(sizeof(Table) + kMaxWarps * kRing));
        if (e != cudaSuccess) return e;
        attr_done[dev] = true;
    }
    const int steps = a.family[0].steps + a.family[1].steps, cuts = (steps + kMaxWarps - 1) / kMaxWarps;
    const int warps = (steps + cuts - 1) / cuts;
    const size_t smem = sizeof(Table) + warps * kRing;
    // as many CTAs as are resident; fewer tokens at a time where that leaves SMs without any
    const int by_registers = 65536 / (kRegisters * 32 * warps), by_smem = int(228 * 1024 / (smem + 1024));
    const int64_t resident = int64_t(num_sms) * (by_registers < by_smem ? by_registers : by_smem) / cuts;
    const int64_t most = resident > 0 ? resident : 1, share = a.batch / most;
    a.tokens = int(share < 1 ? 1 : share > kMost ? kMost : share);
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
