// Decode attention that adds each token's weight to an accumulator (kernels:
// ctx_attn.cuh, mass mode).
#include "ctx_attn.cuh"
#include "../../include/pkv_testing.h"

using namespace pkv;

extern "C" size_t pkv_decode_mass_workspace_size(int32_t batch, int32_t num_q_heads,
                                                 int32_t max_blocks_per_seq,
                                                 const pkv_cache_desc* cache, int32_t num_parts) {
    if (max_blocks_per_seq <= 0) return 0;
    return ctx::workspace_size<ctx::kMass>(batch, num_q_heads, cache, max_blocks_per_seq, num_parts);
}

static pkv_status run_mass(
    const void* q, pkv_dtype q_dtype, const void* k_cache, const void* v_cache,
    const float* k_scales, const float* v_scales, const pkv_cache_desc* cache,
    const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
    int32_t batch, int32_t num_q_heads, float softmax_scale, void* out, const float* mass_in,
    float* mass_out, void* workspace, size_t workspace_bytes, int32_t num_parts,
    uint32_t* dev_status, cudaStream_t stream,
    uint64_t wait_ns, int32_t stall_worker) {
    if (batch > 0 && (!mass_out || !ctx::is_aligned(mass_out, 4) || !ctx::is_aligned(mass_in, 4)))
        return PKV_ERR_INVALID_ARG;
    // the same array, or apart: some threads read while others write
    if (batch > 0 && cache && mass_in && mass_in != mass_out) {
        const double bytes = 64.0 * batch * cache->num_kv_heads * max_blocks_per_seq;
        const uintptr_t x = reinterpret_cast<uintptr_t>(mass_in), y = reinterpret_cast<uintptr_t>(mass_out);
        if (double(x < y ? y - x : x - y) < bytes) return PKV_ERR_INVALID_ARG;
    }
    ctx::Params p = {};
    p.q = q; p.k_cache = k_cache; p.v_cache = v_cache; p.k_scales = k_scales; p.v_scales = v_scales;
    p.block_tables = block_tables; p.context_lens = context_lens;
    p.mass_in = mass_in; p.mass_out = mass_out;
    p.out = out; p.status = dev_status;
    return ctx::run<ctx::kMass>(p, q_dtype, cache, batch, num_q_heads, max_blocks_per_seq,
                                softmax_scale, workspace, workspace_bytes, num_parts, stream,
                                wait_ns, stall_worker);
}

extern "C" pkv_status pkv_decode_attn_mass(
    const void* q, pkv_dtype q_dtype, const void* k_cache, const void* v_cache,
    const float* k_scales, const float* v_scales, const pkv_cache_desc* cache,
    const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
    int32_t batch, int32_t num_q_heads, float softmax_scale, void* out, const float* mass_in,
    float* mass_out, void* workspace, size_t workspace_bytes, int32_t num_parts,
    uint32_t* dev_status, cudaStream_t stream) {
    return run_mass(q, q_dtype, k_cache, v_cache, k_scales, v_scales, cache, block_tables,
        max_blocks_per_seq, context_lens, batch, num_q_heads, softmax_scale, out, mass_in,
        mass_out, workspace, workspace_bytes, num_parts, dev_status, stream, ctx::kWaitLimitNs,
        -1);
}

extern "C" pkv_status pkv_testing_decode_attn_mass_stall(
    const void* q, pkv_dtype q_dtype, const void* k_cache, const void* v_cache,
    const float* k_scales, const float* v_scales, const pkv_cache_desc* cache,
    const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
    int32_t batch, int32_t num_q_heads, float softmax_scale, void* out, const float* mass_in,
    float* mass_out, void* workspace, size_t workspace_bytes, int32_t num_parts,
    uint64_t wait_limit_ns, int32_t stall_worker,
    uint32_t* dev_status, cudaStream_t stream) {
    if (wait_limit_ns > ctx::kWaitLimitNs || stall_worker < -1) return PKV_ERR_INVALID_ARG;
    return run_mass(q, q_dtype, k_cache, v_cache, k_scales, v_scales, cache, block_tables,
        max_blocks_per_seq, context_lens, batch, num_q_heads, softmax_scale, out, mass_in,
        mass_out, workspace, workspace_bytes, num_parts, dev_status, stream, wait_limit_ns,
        stall_worker);
}
