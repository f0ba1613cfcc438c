// attend_coded.cu -- the attention of attend_coded.cuh over the 8-bit formats, and the
// choice among the formats.
#include "attend_coded.cuh"

namespace qsa {

bool attend_coded_shape_supported(int head_dim, int q_heads, int kv_heads)
{
    return (head_dim == 64 || head_dim == 128) && q_heads / kv_heads <= kMaxGqa && kv_heads <= 65535;
}

cudaError_t launch_attend_coded(const AttendCodedArgs &a, cudaStream_t s)
{
    if (a.batch == 0) return cudaSuccess;
    const bool whole = a.ids == nullptr;
    const int runs = coded_max_runs(whole ? a.max_visible / kGroup : (a.row_cap - (kGroup - 1)) / kGroup, whole,
                                    a.q_heads / a.kv_heads);
    const cudaError_t e = is_4bit(a.format) ? launch_attend_coded4(a, runs, s)
                          : a.format == QSA_CODE_INT8 ? launch_format<QSA_CODE_INT8>(a, runs, s)
                                                      : launch_format<QSA_CODE_E4M3>(a, runs, s);
    if (e != cudaSuccess) return e;
    return launch_merge_coded(a, s);
}

}  // namespace qsa
