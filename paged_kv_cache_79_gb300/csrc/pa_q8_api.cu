// extern "C" entry points of the 8-bit cache and of the block tables built on the GPU:
// argument validation, the tensor map and dispatch.  The contract of every function is
// in include/pagedkv.h.
#include <cstring>

#include "pa_internal.h"

using namespace pagedkv;

namespace {

// Sizes every entry point of the cache shares.
pa_status check_sizes(int num_blocks, int max_blocks, int num_kv_heads, int head_dim, int block_size,
                      int dtype)
{
    if (num_blocks <= 0 || max_blocks <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0)
        return PA_ERR_INVALID;
    if (!dtype_ok(dtype) || (head_dim != 64 && head_dim != 128) || (block_size != 16 && block_size != 32))
        return PA_ERR_UNSUPPORTED;
    if ((long long)num_blocks * block_size >= (1ll << 31) || (long long)max_blocks * block_size >= (1ll << 31))
        return PA_ERR_INVALID;
    // (a block then stays below 2^30 bytes, and a run of tokens times its heads below 2^31)
    if (num_kv_heads > 65535)
        return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

// The codes as 4-D: (byte of a 128-byte row, row of a kv head's K and V tiles, kv head,
// block).  One box = one kv head of one block, K tile then V tile, 128-byte swizzle.
bool make_q8_map(CUtensorMap *map, const void *cache, int num_blocks, int B, int Hkv, int D)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc)
        return false;
    const Q8Layout l = q8_layout(B, Hkv, D);
    const cuuint64_t rows = (cuuint64_t)2 * B * D / 128;
    const cuuint64_t dims[4] = {128, rows, (cuuint64_t)Hkv, (cuuint64_t)num_blocks};
    const cuuint64_t strides[3] = {128, rows * 128, (cuuint64_t)l.bytes};
    const cuuint32_t box[4] = {128, (cuuint32_t)rows, 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(cache), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" {

size_t pa_q8_block_bytes(int num_kv_heads, int head_dim, int block_size)
{
    if (check_sizes(1, 1, num_kv_heads, head_dim, block_size, PA_F32) != PA_OK)
        return (size_t)-1;
    return q8_layout(block_size, num_kv_heads, head_dim).bytes;
}

size_t pa_q8_scales_offset(int num_kv_heads, int head_dim, int block_size)
{
    if (check_sizes(1, 1, num_kv_heads, head_dim, block_size, PA_F32) != PA_OK)
        return (size_t)-1;
    return q8_layout(block_size, num_kv_heads, head_dim).scales;
}

pa_status pa_q8_append(const void *k, const void *v, void *kv_cache, const int32_t *block_tables,
                       int max_blocks_per_seq, const int32_t *context_lens, const int32_t *query_start,
                       int num_seqs, int num_tokens, int num_blocks, int num_kv_heads, int head_dim,
                       int block_size, pa_dtype dtype, void *stream)
{
    if (num_seqs == 0 || num_tokens == 0)
        return PA_OK;
    if (!k || !v || !kv_cache || !block_tables || !context_lens || num_seqs < 0 || num_tokens < 0)
        return PA_ERR_INVALID;
    if (!query_start && num_tokens != num_seqs)
        return PA_ERR_INVALID;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(kv_cache, 16) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4) || !aligned(query_start, 4))
        return PA_ERR_INVALID;
    const pa_status st =
        check_sizes(num_blocks, max_blocks_per_seq, num_kv_heads, head_dim, block_size, dtype);
    if (st != PA_OK)
        return st;
    if (num_seqs > kMaxCount || num_tokens > kMaxCount)
        return PA_ERR_UNSUPPORTED;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return cuda_fail(e);
    const Q8Layout l = q8_layout(block_size, num_kv_heads, head_dim);
    Q8AppendParams p;
    p.k = k;
    p.v = v;
    p.cache = static_cast<uint8_t *>(kv_cache);
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.query_start = query_start;
    p.block_bytes = l.bytes;
    p.scales = l.scales;
    p.max_blocks = max_blocks_per_seq;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.num_blocks = num_blocks;
    p.num_kv_heads = num_kv_heads;
    p.block_size = block_size;
    e = launch_q8_append(p, head_dim, dtype, sm_count(dev), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

size_t pa_q8_decode_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                   int block_size, int max_blocks_per_seq)
{
    return pa_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                    max_blocks_per_seq, 0);
}

pa_status pa_q8_decode(void *out, const void *q, const void *kv_cache, const int32_t *block_tables,
                       int max_blocks_per_seq, const int32_t *context_lens, int num_seqs, int num_blocks,
                       float scale, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                       pa_dtype dtype, void *workspace, size_t workspace_bytes, void *stream)
{
    if (num_seqs == 0)
        return PA_OK;
    if (!out || !q || !kv_cache || !block_tables || !context_lens || num_seqs < 0)
        return PA_ERR_INVALID;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4))
        return PA_ERR_INVALID;
    if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0)
        return PA_ERR_INVALID;
    const pa_status st =
        check_sizes(num_blocks, max_blocks_per_seq, num_kv_heads, head_dim, block_size, dtype);
    if (st != PA_OK)
        return st;

    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return cuda_fail(e);
    const int sms = sm_count(dev);
    if (sms <= 0)
        return cuda_fail(cudaErrorNoDevice);
    const size_t need = pa_q8_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                    block_size, max_blocks_per_seq);
    if (need == (size_t)-1 || !workspace || workspace_bytes < need || !aligned(workspace, 16))
        return PA_ERR_INVALID;

    Q8Launch L;
    std::memset(&L, 0, sizeof L);
    DecodeParams &p = L.p;
    p.out = out;
    p.q = q;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    char *const ws = static_cast<char *>(workspace);
    p.counters = reinterpret_cast<unsigned long long *>(ws);
    p.epoch = next_epoch();
    p.part_o = reinterpret_cast<float *>(ws + counter_bytes(sms));
    p.part_lse = reinterpret_cast<float *>(
        ws + counter_bytes(sms) + ((balanced_rows(sms) * (size_t)head_dim * 4 + 255) & ~size_t(255)));
    p.errors = device_error_word(dev, &e);
    if (!p.errors)
        return cuda_fail(e);
    p.wait_ns = wait_limit_ns();
    p.scale_log2 = scale * 1.4426950408889634f;
    p.num_seqs = num_seqs;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = num_q_heads / num_kv_heads;
    p.head_groups = (p.group + kHeadsPerItem - 1) / kHeadsPerItem;
    p.partition_blocks = max_blocks_per_seq;
    p.max_parts = 1;
    p.balanced = 1;
    const Q8Layout l = q8_layout(block_size, num_kv_heads, head_dim);
    L.q8.scales = static_cast<const uint8_t *>(kv_cache) + l.scales;
    L.q8.block_bytes = l.bytes;
    L.head_dim = head_dim;
    L.block_size = block_size;
    L.sm_count = sms;
    if (!make_q8_map(&L.map, kv_cache, num_blocks, block_size, num_kv_heads, head_dim))
        return cuda_fail(cudaErrorInvalidValue);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    e = dtype == PA_F32   ? launch_q8_decode_f32(L, s)
        : dtype == PA_F16 ? launch_q8_decode_f16(L, s)
                          : launch_q8_decode_bf16(L, s);
    return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

pa_status pa_q8_swap_blocks(const void *src_cache, void *dst_cache, const int32_t *src_dst_pairs,
                            int num_pairs, int src_num_blocks, int dst_num_blocks, size_t block_bytes,
                            void *stream)
{
    if (num_pairs == 0)
        return PA_OK;
    if (!src_cache || !dst_cache || !src_dst_pairs || num_pairs < 0 || src_num_blocks <= 0 ||
        dst_num_blocks <= 0 || block_bytes == 0 || block_bytes % 16 != 0)
        return PA_ERR_INVALID;
    if (!aligned(src_cache, 16) || !aligned(dst_cache, 16) || !aligned(src_dst_pairs, 4))
        return PA_ERR_INVALID;
    if (block_bytes / 16 > 65535ull * 1024ull)
        return PA_ERR_UNSUPPORTED;
    if (!device_accessible(src_cache) || !device_accessible(dst_cache) || !device_accessible(src_dst_pairs))
        return PA_ERR_INVALID;
    const cudaError_t e = launch_move_blocks(src_cache, nullptr, dst_cache, nullptr, src_dst_pairs, 2,
                                             src_dst_pairs + 1, 2, num_pairs, src_num_blocks,
                                             dst_num_blocks, block_bytes, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

pa_status pa_q8_copy_blocks(void *kv_cache, const int32_t *src_dst_pairs, int num_pairs, int num_blocks,
                            size_t block_bytes, void *stream)
{
    if (num_pairs == 0)
        return PA_OK;
    if (!kv_cache || !src_dst_pairs || num_pairs < 0 || num_blocks <= 0 || block_bytes == 0 ||
        block_bytes % 16 != 0)
        return PA_ERR_INVALID;
    if (!aligned(kv_cache, 16) || !aligned(src_dst_pairs, 4))
        return PA_ERR_INVALID;
    if (block_bytes / 16 > 65535ull * 1024ull)
        return PA_ERR_UNSUPPORTED;
    const cudaError_t e = launch_move_blocks(kv_cache, nullptr, kv_cache, nullptr, src_dst_pairs, 2,
                                             src_dst_pairs + 1, 2, num_pairs, num_blocks, num_blocks,
                                             block_bytes, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

pa_status pa_build_tables(int32_t *block_tables, int max_blocks_per_seq, int32_t *context_lens_out,
                          const int32_t *context_lens, const int32_t *new_tokens, int num_seqs,
                          int32_t *free_list, int num_blocks, int32_t *num_free_out,
                          const int32_t *num_free, int block_size, int32_t *granted,
                          int32_t *query_start, int64_t *slot_mapping, int num_slots, void *stream)
{
    if (num_seqs < 0 || num_slots < 0 || num_blocks <= 0 || block_size <= 0 || max_blocks_per_seq <= 0)
        return PA_ERR_INVALID;
    if (!free_list || !num_free_out || !num_free || !query_start || (num_slots > 0 && !slot_mapping))
        return PA_ERR_INVALID;
    if (num_seqs > 0 && (!block_tables || !context_lens_out || !context_lens || !new_tokens || !granted))
        return PA_ERR_INVALID;
    for (const void *ptr : {(const void *)block_tables, (const void *)context_lens_out,
                            (const void *)context_lens, (const void *)new_tokens, (const void *)free_list,
                            (const void *)num_free_out, (const void *)num_free, (const void *)granted,
                            (const void *)query_start})
        if (!aligned(ptr, 4))
            return PA_ERR_INVALID;
    if (!aligned(slot_mapping, 8))
        return PA_ERR_INVALID;
    if ((long long)num_blocks * block_size >= (1ll << 31) ||
        (long long)max_blocks_per_seq * block_size >= (1ll << 31))
        return PA_ERR_INVALID;
    if (num_seqs > kMaxCount || num_slots > kMaxCount)
        return PA_ERR_UNSUPPORTED;
    TablesParams p;
    p.block_tables = block_tables;
    p.context_lens_out = context_lens_out;
    p.context_lens = context_lens;
    p.new_tokens = new_tokens;
    p.free_list = free_list;
    p.num_free_out = num_free_out;
    p.num_free = num_free;
    p.granted = granted;
    p.query_start = query_start;
    p.slots = slot_mapping;
    p.max_blocks = max_blocks_per_seq;
    p.num_seqs = num_seqs;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.num_slots = num_slots;
    const cudaError_t e = launch_build_tables(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

}  // extern "C"
