// Decode over the 8-bit paged cache: bf16 queries and outputs.
#include "pa_q8_decode.cuh"

namespace pagedkv {

cudaError_t launch_q8_decode_bf16(const Q8Launch &L, cudaStream_t stream)
{
    return launch_q8_dispatch<__nv_bfloat16>(L, stream);
}

}  // namespace pagedkv
