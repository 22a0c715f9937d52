// Decode attention over a sliding window and sinks (kernels: ctx_attn.cuh,
// window mode).
#include "ctx_attn.cuh"
#include "../../include/pkv_testing.h"

using namespace pkv;

extern "C" size_t pkv_window_decode_workspace_size(int32_t batch, int32_t num_q_heads,
                                                   const pkv_cache_desc* cache,
                                                   int32_t num_parts) {
    return ctx::workspace_size<ctx::kWindow>(batch, num_q_heads, cache, 0, num_parts);
}

static pkv_status run_window(
    const void* q, pkv_dtype q_dtype, const void* k_cache, const void* v_cache,
    const void* k_scales, const void* v_scales, const pkv_cache_desc* cache,
    const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
    int32_t batch, int32_t num_q_heads, float softmax_scale, int32_t window, int32_t num_sinks,
    void* out, void* workspace, size_t workspace_bytes, int32_t num_parts, uint32_t* dev_status,
    cudaStream_t stream, uint64_t wait_ns, int32_t stall_worker) {
    if (window < 0 || num_sinks < 0) return PKV_ERR_INVALID_ARG;
    ctx::Params p = {};
    p.q = q; p.k_cache = k_cache; p.v_cache = v_cache;
    p.k_scales = static_cast<const float*>(k_scales); p.v_scales = static_cast<const float*>(v_scales);
    p.block_tables = block_tables; p.context_lens = context_lens;
    p.window = window; p.sinks = num_sinks;
    p.out = out; p.status = dev_status;
    return ctx::run<ctx::kWindow>(p, q_dtype, cache, batch, num_q_heads, max_blocks_per_seq,
                                  softmax_scale, workspace, workspace_bytes, num_parts, stream,
                                  wait_ns, stall_worker);
}

extern "C" pkv_status pkv_window_decode_attn(
    const void* q, pkv_dtype q_dtype, const void* k_cache, const void* v_cache,
    const void* k_scales, const void* v_scales, const pkv_cache_desc* cache,
    const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
    int32_t batch, int32_t num_q_heads, float softmax_scale, int32_t window, int32_t num_sinks,
    void* out, void* workspace, size_t workspace_bytes, int32_t num_parts, uint32_t* dev_status,
    cudaStream_t stream) {
    return run_window(q, q_dtype, k_cache, v_cache, k_scales, v_scales, cache, block_tables,
        max_blocks_per_seq, context_lens, batch, num_q_heads, softmax_scale, window, num_sinks, out,
        workspace, workspace_bytes, num_parts, dev_status, stream, ctx::kWaitLimitNs, -1);
}

extern "C" pkv_status pkv_testing_window_decode_attn_stall(
    const void* q, pkv_dtype q_dtype, const void* k_cache, const void* v_cache,
    const void* k_scales, const void* v_scales, const pkv_cache_desc* cache,
    const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
    int32_t batch, int32_t num_q_heads, float softmax_scale, int32_t window, int32_t num_sinks,
    void* out, void* workspace, size_t workspace_bytes, int32_t num_parts, uint64_t wait_limit_ns,
    int32_t stall_worker, uint32_t* dev_status, cudaStream_t stream) {
    if (wait_limit_ns > ctx::kWaitLimitNs || stall_worker < -1) return PKV_ERR_INVALID_ARG;
    if (cache && cache->kv_dtype == PKV_U4) return PKV_ERR_UNSUPPORTED;   // waits for nothing that could stay away
    return run_window(q, q_dtype, k_cache, v_cache, k_scales, v_scales, cache, block_tables,
        max_blocks_per_seq, context_lens, batch, num_q_heads, softmax_scale, window, num_sinks, out,
        workspace, workspace_bytes, num_parts, dev_status, stream, wait_limit_ns, stall_worker);
}
