// attend_coded4.cu -- the attention of attend_coded.cuh over the 4-bit formats.
#include "attend_coded.cuh"

namespace qsa {

cudaError_t launch_attend_coded4(const AttendCodedArgs &a, int runs, cudaStream_t s)
{
    return a.format == QSA_CODE_INT4 ? launch_format<QSA_CODE_INT4>(a, runs, s) : launch_format<QSA_CODE_E2M1>(a, runs, s);
}

}  // namespace qsa
