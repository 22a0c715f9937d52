// Decode attention over chosen blocks (kernels: ctx_attn.cuh, list mode).
#include "ctx_attn.cuh"
#include "../../include/pkv_testing.h"

using namespace pkv;

extern "C" size_t pkv_sparse_decode_workspace_size(int32_t batch, int32_t num_q_heads,
                                                   const pkv_cache_desc* cache,
                                                   int32_t num_parts) {
    return ctx::workspace_size<ctx::kList>(batch, num_q_heads, cache, 0, num_parts);
}

static pkv_status run_sparse(
    const void* q, pkv_dtype q_dtype, const void* k_cache, const void* v_cache,
    const float* k_scales, const float* v_scales, const pkv_cache_desc* cache,
    const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
    const int32_t* block_lists, int32_t max_list, const int32_t* list_lens, int32_t batch,
    int32_t num_q_heads, float softmax_scale, void* out, void* workspace, size_t workspace_bytes,
    int32_t num_parts, uint32_t* dev_status, cudaStream_t stream,
    uint64_t wait_ns, int32_t stall_worker) {
    if (max_list < 0) return PKV_ERR_INVALID_ARG;
    if (batch > 0) {
        if (!list_lens || !ctx::is_aligned(list_lens, 4)) return PKV_ERR_INVALID_ARG;
        if (max_list > 0 && (!block_lists || !ctx::is_aligned(block_lists, 4)))
            return PKV_ERR_INVALID_ARG;
        if ((long long)batch * max_list > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
    }
    ctx::Params p = {};
    p.q = q; p.k_cache = k_cache; p.v_cache = v_cache; p.k_scales = k_scales; p.v_scales = v_scales;
    p.block_tables = block_tables; p.context_lens = context_lens;
    p.lists = block_lists; p.list_lens = list_lens; p.max_list = max_list;
    p.out = out; p.status = dev_status;
    return ctx::run<ctx::kList>(p, q_dtype, cache, batch, num_q_heads, max_blocks_per_seq,
                                softmax_scale, workspace, workspace_bytes, num_parts, stream,
                                wait_ns, stall_worker);
}

extern "C" pkv_status pkv_sparse_decode_attn(
    const void* q, pkv_dtype q_dtype, const void* k_cache, const void* v_cache,
    const float* k_scales, const float* v_scales, const pkv_cache_desc* cache,
    const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
    const int32_t* block_lists, int32_t max_list, const int32_t* list_lens, int32_t batch,
    int32_t num_q_heads, float softmax_scale, void* out, void* workspace, size_t workspace_bytes,
    int32_t num_parts, uint32_t* dev_status, cudaStream_t stream) {
    return run_sparse(q, q_dtype, k_cache, v_cache, k_scales, v_scales, cache, block_tables,
        max_blocks_per_seq, context_lens, block_lists, max_list, list_lens, batch, num_q_heads,
        softmax_scale, out, workspace, workspace_bytes, num_parts, dev_status, stream,
        ctx::kWaitLimitNs, -1);
}

extern "C" pkv_status pkv_testing_sparse_decode_attn_stall(
    const void* q, pkv_dtype q_dtype, const void* k_cache, const void* v_cache,
    const float* k_scales, const float* v_scales, const pkv_cache_desc* cache,
    const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
    const int32_t* block_lists, int32_t max_list, const int32_t* list_lens, int32_t batch,
    int32_t num_q_heads, float softmax_scale, void* out, void* workspace, size_t workspace_bytes,
    int32_t num_parts, uint64_t wait_limit_ns, int32_t stall_worker,
    uint32_t* dev_status, cudaStream_t stream) {
    if (wait_limit_ns > ctx::kWaitLimitNs || stall_worker < -1) return PKV_ERR_INVALID_ARG;
    return run_sparse(q, q_dtype, k_cache, v_cache, k_scales, v_scales, cache, block_tables,
        max_blocks_per_seq, context_lens, block_lists, max_list, list_lens, batch, num_q_heads,
        softmax_scale, out, workspace, workspace_bytes, num_parts, dev_status, stream,
        wait_limit_ns, stall_worker);
}
