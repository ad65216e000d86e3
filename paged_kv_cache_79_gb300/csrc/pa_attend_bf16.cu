// pa_attend for bf16: the tcgen05 kernel.
#include "pa_attend_tc.cuh"

namespace pagedkv {

cudaError_t launch_attend_bf16(const AttendLaunch &L, cudaStream_t stream)
{
    return tc::launch_type<__nv_bfloat16>(L, stream);
}

}  // namespace pagedkv
