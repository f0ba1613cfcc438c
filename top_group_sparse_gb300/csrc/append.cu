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
// Layout.  A lane holds four neighbouring dims, so a head is a quarter of its width in
// lanes (a warp takes 1, 2 or 4 heads at once) and every access is a 16-byte (or, of
// 16-bit types, 8-byte) piece of a row.  The partner of a dim is in the same lane
// (neighbours) or in another at a fixed distance (halves: dims is a multiple of 8), so a
// rotation is z = y * cos + partner * (+-sin) everywhere.  A warp takes consecutive heads
// of one token and computes its sines once for all of them: all the heads of a token when
// there are enough tokens to fill the GPU, else as few as one step.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache_internal.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 6;
constexpr int kWarpsWanted = 64;      // tasks per SM below which a token's heads are spread over more warps
constexpr int kMaxPairs = 64;

struct Table {
    uint64_t turns[2][QSA_MAX_AXES][kMaxPairs];  // by family: heads of d, heads of d_I
    float bad[2][kMaxPairs];                     // NaN for a pair with a frequency out of range, else 0
};

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

template <typename T>
struct Raw { using type = uint2; };
template <>
struct Raw<float> { using type = float4; };

template <typename T>
__device__ __forceinline__ float4 widen(typename Raw<T>::type r)
{
    if constexpr (sizeof(T) == 4) {
        return r;
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u), __uint_as_float(r.y << 16),
                           __uint_as_float(r.y & 0xffff0000u));
    } else {
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&r.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&r.y));
        return make_float4(a.x, a.y, b.x, b.y);
    }
}

// Heads [step * (128/W), ..) of one family of token b, `steps` steps of them, by a warp.
template <typename T, int W, int kFamily>
__device__ __forceinline__ void append_heads(const AppendArgs &a, const Table &table, int b, int step, int steps)
{
    constexpr int kLanes = W / 4, kRows = 32 / kLanes;
    const int lane = threadIdx.x & 31, l = lane % kLanes, sub = lane / kLanes;
    const AppendFamily &f = a.family[kFamily];
    using R = typename Raw<T>::type;

    // the row's head, by the order q, k, v (q_idx, idx_key)
    auto part_of = [&](int head, int &at) {
        int k = 0;
        at = head;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (at >= f.heads[i] && k == i) {
                at -= f.heads[i];
                k = i + 1;
            }
        return k;
    };
    auto load = [&](int s) {
        const int head = (step + s) * kRows + sub;
        R r{};
        if (s < steps && head < f.all_heads) {
            int at;
            const int k = part_of(head, at);
            r = __ldg(reinterpret_cast<const R *>(static_cast<const T *>(f.rows[k]) + b * f.stride[k] + at * W) + l);
        }
        return r;
    };
    R next = load(0);

    // where the token goes
    const int vis = __ldg(a.visible + b);
    const bool in_range = vis >= 0 && vis <= a.max_visible;
    if (vis == 0) return;
    int64_t row = -1;  // of the caches, or of idx_keys
    if (!in_range) {
        if (step == 0 && lane == 0) set_error(a.err, QSA_DEVERR_VISIBLE_RANGE);
    } else if constexpr (kFamily == 0) {
        if (f.heads[1] + f.heads[2] > 0) {
            const int slot = __ldg(a.slot_map + __ldg(a.slot_offset + b) + vis - 1);
            if (slot >= 0 && slot < a.num_slots) row = slot;
            else if (step == 0 && lane == 0) set_error(a.err, QSA_DEVERR_SLOT_RANGE);
        }
    } else {
        if (f.heads[1] > 0) row = __ldg(a.key_offset + b) + vis - 1;
    }

    // this lane's four dims: cos, and the factor of their partners
    const int half = f.dims / 2;
    const bool turned = 4 * l < f.dims;
    int partner = lane;
    float c[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    if (f.dims > 0) {
        const bool second = 4 * l >= half;
        if (!f.neighbours && turned) partner = second ? lane - half / 4 : lane + half / 4;
        const int j0 = !turned ? 0 : f.neighbours ? 2 * l : second ? 4 * l - half : 4 * l;
        const int n = f.neighbours ? 2 : 4;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (u >= n) break;
            uint64_t phase = 0;
            for (int x = 0; x < a.axes; ++x)
                phase += uint64_t(int64_t(__ldg(a.positions + int64_t(x) * a.batch + b))) * table.turns[kFamily][x][j0 + u];
            float s0, c0;
            sincospif(float(int32_t(phase >> 32)) * 0x1p-31f, &s0, &c0);  // half turns
            c[u] = c0 + table.bad[kFamily][j0 + u];
            sn[u] = s0 + table.bad[kFamily][j0 + u];
        }
        if (f.neighbours) {
            c[3] = c[2] = c[1];
            sn[3] = sn[1];
            sn[2] = -sn[1];
            c[1] = c[0];
            sn[1] = sn[0];
            sn[0] = -sn[0];
        } else if (!second) {
#pragma unroll
            for (int u = 0; u < 4; ++u) sn[u] = -sn[u];
        }
    }

    for (int s = 0; s < steps; ++s) {
        const R raw = next;
        next = load(s + 1);
        const int head = (step + s) * kRows + sub;
        int at;
        const int k = part_of(head, at);
        const bool some = head < f.all_heads;
        float4 x = widen<T>(raw);
        if (f.any_norm) {
            float ss = fmaf(x.x, x.x, fmaf(x.y, x.y, fmaf(x.z, x.z, x.w * x.w)));
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (some && f.norm[k] != nullptr) {
                const float4 w = __ldg(reinterpret_cast<const float4 *>(f.norm[k]) + l);
                const float r = __frsqrt_rn(fmaf(ss, 1.0f / W, a.eps));
                x = make_float4(x.x * r * w.x, x.y * r * w.y, x.z * r * w.z, x.w * r * w.w);
            }
        }
        if (f.dims > 0) {
            float4 p;
            if (f.neighbours) {
                p = make_float4(x.y, x.x, x.w, x.z);
            } else {
                p.x = __shfl_sync(0xffffffffu, x.x, partner);
                p.y = __shfl_sync(0xffffffffu, x.y, partner);
                p.z = __shfl_sync(0xffffffffu, x.z, partner);
                p.w = __shfl_sync(0xffffffffu, x.w, partner);
            }
            if (turned && !(kFamily == 0 && k == 2))
                x = make_float4(fmaf(x.x, c[0], p.x * sn[0]), fmaf(x.y, c[1], p.y * sn[1]), fmaf(x.z, c[2], p.z * sn[2]),
                                fmaf(x.w, c[3], p.w * sn[3]));
        }
        if (!some) continue;
        if (k == 0) {  // the batch's own rows; zeros for a query that is out of range
            if (!in_range) x = make_float4(0.f, 0.f, 0.f, 0.f);
            *(reinterpret_cast<float4 *>(f.out[0] + (int64_t(b) * f.heads[0] + at) * W) + l) = x;
        } else if (row >= 0) {
            *(reinterpret_cast<float4 *>(f.out[k] + (row * f.out_heads + at) * W) + l) = x;
        }
    }
}

template <typename T, int D, int DI>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) append_kernel(const __grid_constant__ AppendArgs a)
{
    __shared__ Table table;
    const int tid = threadIdx.x, warp = tid >> 5;
    wait_for_predecessor();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int pairs = a.family[i].dims / 2;
        for (int j = tid; j < pairs; j += kThreads) {
            float bad = 0.0f;
            for (int x = 0; x < a.axes; ++x) {
                const float f = __ldg(a.family[i].freq + x * pairs + j);
                const bool ok = fabsf(f) < 65536.0f;
                table.turns[i][x][j] = ok ? turns_of(f) : 0;
                if (!ok) bad = __int_as_float(0x7fffffff);
            }
            table.bad[i][j] = bad;
        }
    }
    __syncthreads();
    const int64_t tasks = int64_t(a.batch) * a.tasks;
    for (int64_t t = int64_t(blockIdx.x) * kWarps + warp; t < tasks; t += int64_t(gridDim.x) * kWarps) {
        const int b = int(t / a.tasks), k = int(t - int64_t(b) * a.tasks);
        if (k < a.family[0].tasks) {
            append_heads<T, D, 0>(a, table, b, k * a.steps, min(a.steps, a.family[0].steps - k * a.steps));
        } else {
            const int i = k - a.family[0].tasks;
            append_heads<T, DI, 1>(a, table, b, i * a.steps, min(a.steps, a.family[1].steps - i * a.steps));
        }
    }
}

template <typename T>
cudaError_t launch_t(const AppendArgs &a, int d, int idx, int num_sms, cudaStream_t s)
{
    const int64_t ctas = (int64_t(a.batch) * a.tasks + kWarps - 1) / kWarps, most = int64_t(num_sms) * kCtasPerSm;
    auto launch = [&](void (*kernel)(const AppendArgs)) {
        return launch_kernel(kernel, dim3(unsigned(ctas < most ? ctas : most)), dim3(kThreads), 0, s, true, a);
    };
    if (d == 128) return launch(idx == 64 ? append_kernel<T, 128, 64> : append_kernel<T, 128, 32>);
    return launch(idx == 64 ? append_kernel<T, 64, 64> : append_kernel<T, 64, 32>);
}

}  // namespace

cudaError_t launch_append(AppendArgs a, int type, int d, int idx, int num_sms, cudaStream_t s)
{
    if (a.batch == 0) return cudaSuccess;
    auto cut = [&](int steps) {
        a.steps = steps;
        a.tasks = 0;
        for (AppendFamily &f : a.family) a.tasks += f.tasks = (f.steps + steps - 1) / steps;
    };
    int most = 0;
    for (int i = 0; i < 2; ++i) {
        AppendFamily &f = a.family[i];
        const int rows = 128 / (i == 0 ? d : idx);
        f.all_heads = f.heads[0] + f.heads[1] + f.heads[2];
        f.steps = (f.all_heads + rows - 1) / rows;
        most = f.steps > most ? f.steps : most;
    }
    for (cut(most); a.steps > 1 && int64_t(a.batch) * a.tasks < int64_t(num_sms) * kWarpsWanted;) cut((a.steps + 1) / 2);
    if (type == QSA_ROWS_F32) return launch_t<float>(a, d, idx, num_sms, s);
    if (type == QSA_ROWS_BF16) return launch_t<__nv_bfloat16>(a, d, idx, num_sms, s);
    return launch_t<__half>(a, d, idx, num_sms, s);
}

}  // namespace qsa
