// pa_attend for f16: the tcgen05 kernel.
#include "pa_attend_tc.cuh"

namespace pagedkv {

cudaError_t launch_attend_f16(const AttendLaunch &L, cudaStream_t stream)
{
    return tc::launch_type<__half>(L, stream);
}

}  // namespace pagedkv
