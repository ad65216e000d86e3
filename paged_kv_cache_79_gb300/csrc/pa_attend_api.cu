// extern "C" entry points of pa_attend: argument validation, workspace, tensor maps and
// dispatch.  The contract is in include/pagedkv.h.
#include <cstring>

#include "pa_attend.cuh"

using namespace pagedkv;

namespace {

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

bool attend_sizes_ok(int num_q_heads, int num_kv_heads, int head_dim)
{
    return num_q_heads > 0 && num_kv_heads > 0 && num_q_heads % num_kv_heads == 0 &&
           (head_dim == 64 || head_dim == 128);
}

struct Workspace {
    size_t ml, o, bytes;  // offsets of the partial rows, the whole
};
Workspace workspace_of(int ctas, int part_rows, int head_dim)
{
    Workspace w;
    const size_t rows = (size_t)ctas * 2 * part_rows;
    w.ml = up256((size_t)ctas * sizeof(AttendCut));
    w.o = w.ml + up256(rows * sizeof(float2));
    w.bytes = w.o + up256(rows * head_dim * sizeof(float));
    return w;
}

CUtensorMapDataType type_of(int dtype)
{
    return dtype == PA_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

// A 16-bit cache [num_blocks][B][Hkv][d] as (64 elements, token slot, column of 64, kv head); a
// box is `columns` columns of a block's rows of one kv head, each B rows of 128 bytes, 128-byte
// swizzle.
bool make_blocks_map(CUtensorMap *map, const void *cache, int num_blocks, int B, int Hkv, int D, int columns,
                     int dtype)
{
    const EncodeTiledFn enc = encode_fn();
    if (!enc)
        return false;
    const cuuint64_t dims[4] = {64, (cuuint64_t)num_blocks * B, (cuuint64_t)D / 64, (cuuint64_t)Hkv};
    const cuuint64_t strides[3] = {(cuuint64_t)Hkv * D * 2, 128, (cuuint64_t)D * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)B, (cuuint32_t)columns, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, type_of(dtype), 4, const_cast<void *>(cache), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of queries as (64 elements, head, token, column of 64); a box is one column of `heads`
// heads of `tokens` tokens: a row tile's rows in their order.
bool make_rows_map(CUtensorMap *map, const void *q, long long stride, int num_tokens, int Hq, int D, int heads,
                   int tokens, int dtype)
{
    const EncodeTiledFn enc = encode_fn();
    if (!enc)
        return false;
    const cuuint64_t dims[4] = {64, (cuuint64_t)Hq, (cuuint64_t)num_tokens, (cuuint64_t)D / 64};
    const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2, 128};
    const cuuint32_t box[4] = {64, (cuuint32_t)heads, (cuuint32_t)tokens, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, type_of(dtype), 4, const_cast<void *>(q), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" {

size_t pa_attend_workspace_size(int num_q_heads, int num_kv_heads, int head_dim)
{
    if (!attend_sizes_ok(num_q_heads, num_kv_heads, head_dim))
        return (size_t)-1;
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) {
        cudaGetLastError();
        return (size_t)-1;
    }
    const int sms = sm_count(device);
    return sms > 0 ? workspace_of(sms, kAttendRows, head_dim).bytes : (size_t)-1;
}

pa_status pa_attend(void *out, float *lse, const void *q, long long q_stride, const void *k_cache,
                    const void *v_cache, const int32_t *block_tables, int max_blocks_per_seq,
                    const int32_t *context_lens, const int32_t *query_start, int num_seqs, int num_tokens,
                    int num_blocks, float scale, int causal, int num_q_heads, int num_kv_heads, int head_dim,
                    int block_size, pa_dtype dtype, void *workspace, size_t workspace_bytes, void *stream)
{
    if (num_seqs == 0 || num_tokens == 0)
        return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start || num_seqs < 0 ||
        num_tokens < 0)
        return PA_ERR_INVALID;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(query_start, 4) || !aligned(lse, 4))
        return PA_ERR_INVALID;
    if (num_blocks <= 0 || max_blocks_per_seq <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
        num_q_heads % num_kv_heads != 0)
        return PA_ERR_INVALID;
    if (!dtype_ok(dtype) || (head_dim != 64 && head_dim != 128) || (block_size != 16 && block_size != 32))
        return PA_ERR_UNSUPPORTED;
    if ((long long)num_blocks * block_size >= (1ll << 31) || (long long)max_blocks_per_seq * block_size >= (1ll << 31))
        return PA_ERR_INVALID;
    const long long q_row = (long long)num_q_heads * head_dim;
    if (num_tokens > 1 && (q_stride < q_row || q_stride % (dtype == PA_F32 ? 4 : 8) != 0))
        return PA_ERR_INVALID;
    if (num_seqs > kMaxCount || num_tokens > kMaxCount || num_q_heads > 65535 || q_stride >= (1ll << 36))
        return PA_ERR_UNSUPPORTED;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess)
        return cuda_fail(e);
    const int sms = sm_count(device);
    if (sms <= 0)
        return cuda_fail(cudaErrorNoDevice);
    const size_t need = workspace_of(sms, kAttendRows, head_dim).bytes;
    if (!workspace || workspace_bytes < need || !aligned(workspace, 16))
        return PA_ERR_INVALID;

    AttendLaunch L;
    std::memset(&L, 0, sizeof L);
    AttendParams &p = L.p;
    p.out = out;
    p.lse = lse;
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.query_start = query_start;
    p.q_stride = num_tokens > 1 ? q_stride : q_row;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.num_seqs = num_seqs;
    p.num_rows = num_tokens;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = num_q_heads / num_kv_heads;
    p.causal = causal != 0;
    p.errors = device_error_word(device, &e);
    if (!p.errors)
        return cuda_fail(e);
    p.wait_ns = wait_limit_ns();
    L.head_dim = head_dim;
    // fp32: items of kF32TileRows rows, two CTAs per SM; fp16 and bf16: two tiles of 128 rows, one
    // CTA per SM.  Either way at most two slots of kAttendRows rows per SM.
    const bool f32 = dtype == PA_F32;
    const int tile = f32 ? kF32TileRows : kAttendRows / 2;
    p.heads_per_item = p.group < tile ? p.group : tile;
    p.head_chunks = (p.group + p.heads_per_item - 1) / p.heads_per_item;
    p.units = num_kv_heads * p.head_chunks;
    p.tokens_per_item = tile / p.heads_per_item * (f32 ? 1 : 2);
    p.few_tokens = f32 ? 0 : p.tokens_per_item / 2;
    p.part_rows = f32 ? kF32TileRows : kAttendRows;
    L.ctas = f32 ? 2 * sms : sms;
    if (!f32 &&
        (!make_rows_map(&L.map_q, q, p.q_stride, num_tokens, num_q_heads, head_dim, p.heads_per_item,
                        p.tokens_per_item / 2, dtype) ||
         !make_blocks_map(&L.map_k, k_cache, num_blocks, block_size, num_kv_heads, head_dim, 1, dtype) ||
         !make_blocks_map(&L.map_v, v_cache, num_blocks, block_size, num_kv_heads, head_dim, head_dim / 64, dtype)))
        return cuda_fail(cudaErrorInvalidValue);
    const Workspace w = workspace_of(L.ctas, p.part_rows, head_dim);
    char *const ws = static_cast<char *>(workspace);
    p.cuts = reinterpret_cast<AttendCut *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(ws + w.ml);
    p.part_o = reinterpret_cast<float *>(ws + w.o);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    e = dtype == PA_F32 ? launch_attend_f32(L, s) : dtype == PA_F16 ? launch_attend_f16(L, s) : launch_attend_bf16(L, s);
    if (e == cudaSuccess)
        e = launch_attend_merge(L, dtype, s);
    return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

}  // extern "C"
