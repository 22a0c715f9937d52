// Multi-query paged attention: the host side of pkv_multiquery_attn and
// pkv_window_multiquery_attn (the mma.sync split kernel and its combine live in
// mq_split.cuh, the tcgen05 kernel for long query runs in mq_tc.cuh).
#include <cuda.h>

#include <mutex>

#include "mq_tc.cuh"
#include "mq_wide.cuh"

namespace pkv {
namespace {

// ------------------------------------------------------------------- host ---
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(f);
    });
    return fn;
}

// The cache as a 2-D tensor [rows = NB * Hkv * 16][D] of 16-bit values, read
// in 16 x 64 boxes with the 128-byte swizzle.
bool encode_cache_map(CUtensorMap* m, const void* base, bool bf16, int D, long long rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {cuuint64_t(D), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(D) * 2};
    const cuuint32_t box[2] = {64, 16};
    const cuuint32_t es[2] = {1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
              const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// INT8 cache [rows, 128] of byte codes as 16 x 128-byte boxes, 128-byte swizzle.
bool encode_i8_map(CUtensorMap* m, const void* base, long long rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {128, cuuint64_t(rows)};
    const cuuint64_t strides[1] = {128};
    const cuuint32_t box[2] = {128, 16};
    const cuuint32_t es[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// With a window, runs of more rows than this may take the wide-chunk tcgen05 kernel
// (mq_wide.cuh), whose time hardly depends on them up to a tile of 128: windows of 4096 of 64
// sequences, 8 kv heads, bf16: 32 rows split 216 us, 36 rows wide 274 (split 435),
// 64 rows 275 and 453, 128 rows 280 and 882.
constexpr int kWideMin = 32;

// Whether they do: that kernel leaves a pair of tiles to one SM, which walks its chunks one
// after another; the split kernel has every SM at work whatever the sizes. Estimates of both
// in us, fitted to 1 to 512 segments (sequences x kv heads) of 36 to 4800 rows, 4 heads a
// group, windows of 512 and 4096, for every type and head_dim; of the two they choose one
// that is 1 % slower than the better on average and 23 % at worst. Measured, wide and split:
//   window, segments, rows   bf16 D 128    bf16 D 64     INT8, fp16 q, D 128   D 64
//   4096     8    64          68   22      57   19          80   25            64   22
//   4096     8   512         103   74      99   47         131  100           116   55
//   4096    16   512         103  128     100   79         132  181           116   91
//   4096    64   128          73  127      61   77          84  178            69   90
//    512    64    64          17   25      16   18          22   28            18   22
//    512     8   256          25   21      22   17          31   24            25   20
//    512     1  4800          25   48      23   41          32   54            26   46
// (fp16 caches are as bf16 ones within 3 %.) `blocks`: the most that a pair of tiles sees.
// bf16 queries over INT8 take it in any case: it scales their rows, which may have any size
// there.
struct WideCost {
    double start, tile, pair;      // wide: us, us per chunk of one tile and of two
    double begin, block, rows;     // split: us, us per block of a segment's 64 rows, per 64 rows
};
bool wide_pays(const pkv_cache_desc* c, pkv_dtype q_dtype, long long segs, long long rows, long long blocks) {
    const bool codes = c->kv_dtype == PKV_I8, wide_rows = c->head_dim == 128;
    if (rows <= kWideMin) return false;
    if (codes && q_dtype == PKV_BF16) return true;
    static const WideCost costs[2][2] = {{{7.5, 1.65, 3.0, 15, 2.0e-3, 0.25}, {8.2, 1.92, 3.3, 16, 3.5e-3, 0.2}},
                                         {{8.0, 2.0, 3.5, 16, 2.3e-3, 0.25}, {10, 2.5, 4.3, 16, 5.0e-3, 0.25}}};
    const WideCost& t = costs[codes][wide_rows];
    const long long rounds = (segs * ((rows + 255) / 256) + 151) / 152, chunks = (blocks + 7) / 8;
    const double wide = t.start + double(rounds) * double(chunks) * (rows <= kTcRows ? t.tile : t.pair);
    const double tiles = double((rows + 63) / 64);
    return wide < t.begin + (t.block * double(segs) * double(blocks) + t.rows) * tiles;
}

// Query rows per (sequence, kv head) up to which fp16 / bf16 caches take the
// short-run kernel (mq_t.cu).
constexpr long long kMqtMaxRows = 24;

struct MqPlan {
    MqOps ops;
    int G, nw, tmax;
    long long workers;
    size_t smem, ws_prefix, ws_ml, ws_o, ws_total;
};

bool mq_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t mq_align256(size_t x) { return (x + 255) & ~size_t(255); }

// Checks the sizes and picks the kernel, tile height, workers and workspace.
// `win`: pkv_window_multiquery_attn's kernels.
pkv_status mq_plan(const pkv_cache_desc* c, int batch, int hq, int max_q, pkv_dtype q_dtype,
                   int num_parts, MqPlan* pl, bool win = false) {
    if (!c || c->num_blocks <= 0 || c->num_kv_heads <= 0 || c->head_dim <= 0)
        return PKV_ERR_INVALID_ARG;
    if (batch < 0 || hq <= 0 || hq % c->num_kv_heads || max_q <= 0 || num_parts < 0)
        return PKV_ERR_INVALID_ARG;
    if (c->kv_dtype != PKV_BF16 && c->kv_dtype != PKV_F16 && c->kv_dtype != PKV_I8)
        return PKV_ERR_INVALID_ARG;
    if (q_dtype != PKV_BF16 && q_dtype != PKV_F16) return PKV_ERR_INVALID_ARG;
    if (c->kv_dtype != PKV_I8 && q_dtype != c->kv_dtype) return PKV_ERR_INVALID_ARG;
    if (c->block_size != kBlockSize || batch > kMqMaxBatch) return PKV_ERR_UNSUPPORTED;
    if ((long long)c->num_blocks * c->num_kv_heads * kBlockSize >= (1LL << 31))
        return PKV_ERR_UNSUPPORTED;
    pl->G = hq / c->num_kv_heads;
    const long long rows = (long long)max_q * pl->G;
    if (rows > (1LL << 24)) return PKV_ERR_UNSUPPORTED;
    pl->nw = rows <= 16 ? 1 : (rows <= 32 ? 2 : 4);
    // short runs: rows on the MMA's N side, a warp per worker (INT8: head_dim 128)
    bool ok = rows <= kMqtMaxRows && (win ? mqt_pick_win : mqt_pick)(
        c->kv_dtype, q_dtype, c->head_dim, pl->G, int((rows + 7) / 8), &pl->ops);
    if (!ok && win)
        ok = c->kv_dtype == PKV_I8 ? mq_pick_win_i8(q_dtype, c->head_dim, pl->G, pl->nw, &pl->ops)
                                   : mq_pick_win(c->kv_dtype, c->head_dim, pl->G, pl->nw, &pl->ops);
    else if (!ok && c->kv_dtype == PKV_I8)
        ok = mq_pick_i8(q_dtype, c->head_dim, pl->G, pl->nw, &pl->ops);
    else if (!ok)
        ok = c->kv_dtype == PKV_BF16 ? mq_pick_d<BF16, BF16>(c->head_dim, pl->G, pl->nw, &pl->ops)
                                     : mq_pick_d<F16, F16>(c->head_dim, pl->G, pl->nw, &pl->ops);
    if (!ok) return PKV_ERR_UNSUPPORTED;
    pl->tmax = int((rows + pl->ops.rt - 1) / pl->ops.rt);
    pl->smem = size_t(pl->ops.fixed_smem) + 4 * size_t((batch < 1 ? 1 : batch) + 1);
    if (num_parts > 0) {
        pl->workers = num_parts;
    } else {
        int dev = 0, sms = 0, blocks = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            pl->ops.occupancy(&blocks, pl->smem) != cudaSuccess || blocks <= 0)
            return PKV_ERR_CUDA;
        pl->workers = (long long)sms * blocks * pl->ops.wpc;
    }
    const long long slots = (long long)batch * c->num_kv_heads * pl->tmax + pl->workers;
    pl->ws_prefix = 0;
    pl->ws_ml = mq_align256(sizeof(int32_t) * size_t(batch + 1));
    pl->ws_o = pl->ws_ml + mq_align256(size_t(slots) * pl->ops.rt * 2 * sizeof(float));
    pl->ws_total = pl->ws_o + mq_align256(size_t(slots) * pl->ops.rt * c->head_dim * sizeof(float));
    return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

static size_t mq_workspace(int batch, int hq, int max_q, const pkv_cache_desc* cache, int num_parts,
                           bool win) {
    if (!cache) return 0;
    // over INT8 for either type of q: their kernels' registers, and so their workers, differ
    size_t most = 0;
    for (pkv_dtype qd : {PKV_BF16, PKV_F16}) {
        MqPlan pl;
        if (cache->kv_dtype != PKV_I8) qd = cache->kv_dtype;
        if (mq_plan(cache, batch, hq, max_q, qd, num_parts, &pl, win) != PKV_OK) return 0;
        most = std::max(most, pl.ws_total);
        if (cache->kv_dtype != PKV_I8) break;
    }
    return most;
}

extern "C" size_t pkv_multiquery_workspace_size(int32_t batch, int32_t num_q_heads,
                                                int32_t max_q_len, const pkv_cache_desc* cache,
                                                int32_t num_parts) {
    return mq_workspace(batch, num_q_heads, max_q_len, cache, num_parts, false);
}

extern "C" size_t pkv_window_multiquery_workspace_size(int32_t batch, int32_t num_q_heads,
                                                       int32_t max_q_len,
                                                       const pkv_cache_desc* cache,
                                                       int32_t num_parts) {
    return mq_workspace(batch, num_q_heads, max_q_len, cache, num_parts, true);
}

namespace {

constexpr uint64_t kTcWaitNs = 2000000000ull;

// The tcgen05 launcher that serves runs of max_q rows per query head group
// over this cache (16-bit caches, rows filling 128-row tiles), or nullptr;
// q and out must also be 16-byte aligned.
TcLaunch tc_for(const pkv_cache_desc* cache, int max_q, int G) {
    if (cache->kv_dtype == PKV_I8 || (long long)max_q * G < kTcRows) return nullptr;
    return cache->kv_dtype == PKV_BF16 ? tc_pick<BF16>(cache->head_dim, G)
                                       : tc_pick<F16>(cache->head_dim, G);
}

// The wide-chunk launcher where it serves pkv_window_multiquery_attn, or nullptr; q and out
// must also be 16-byte aligned.
WideLaunch wide_for(const pkv_cache_desc* cache, pkv_dtype q_dtype, int batch, int max_q, int G, int mb,
                    int window, int sinks) {
    const long long span = std::min(max_q, 2 * kTcRows / G);             // queries of a pair of tiles
    const long long seen = (window + span) / kBlockSize + 2 + ((long long)sinks + kBlockSize - 1) / kBlockSize;
    if (!wide_pays(cache, q_dtype, (long long)batch * cache->num_kv_heads, (long long)max_q * G,
                   window ? std::min<long long>(mb, seen) : mb))
        return nullptr;
    return cache->kv_dtype == PKV_I8 ? wide_pick_i8(q_dtype, cache->head_dim, G)
                                     : wide_pick(cache->kv_dtype, cache->head_dim, G);
}

pkv_status run_multiquery(const void* q, pkv_dtype q_dtype, const int32_t* cu_q,
                          int32_t max_q_len, const void* k_cache, const void* v_cache,
                          const float* k_scales, const float* v_scales,
                          const pkv_cache_desc* cache, const int32_t* block_tables,
                          int32_t max_blocks_per_seq, const int32_t* context_lens, int32_t batch,
                          int32_t num_q_heads, float softmax_scale, void* out, void* workspace,
                          size_t workspace_bytes, int32_t num_parts, uint32_t* dev_status,
                          cudaStream_t stream, uint64_t wait_ns, int stall_cta, bool win = false,
                          int window = 0, int sinks = 0) {
    MqPlan pl;
    pkv_status s = mq_plan(cache, batch, num_q_heads, max_q_len, q_dtype, num_parts, &pl, win);
    if (s != PKV_OK) return s;
    if (batch == 0) return PKV_OK;
    if (!q || !cu_q || !k_cache || !v_cache || !block_tables || !context_lens || !out)
        return PKV_ERR_INVALID_ARG;
    if (!mq_aligned(q, 4) || !mq_aligned(out, 4) || !mq_aligned(k_cache, 16) ||
        !mq_aligned(v_cache, 16) || !mq_aligned(cu_q, 4) || !mq_aligned(block_tables, 4) ||
        !mq_aligned(context_lens, 4) || (dev_status && !mq_aligned(dev_status, 4)))
        return PKV_ERR_INVALID_ARG;
    if (max_blocks_per_seq <= 0 || max_blocks_per_seq > 0x7fffffff / kBlockSize ||
        !(softmax_scale == softmax_scale) || softmax_scale > 3.0e38f ||
        softmax_scale < -3.0e38f || pl.workers > 0x7fffffffLL)
        return PKV_ERR_INVALID_ARG;
    const bool i8 = cache->kv_dtype == PKV_I8;
    if (i8 && (!k_scales || !v_scales || !mq_aligned(k_scales, 4) || !mq_aligned(v_scales, 4) ||
               !mq_aligned(q, 16)))
        return PKV_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < pl.ws_total || !mq_aligned(workspace, 256))
        return PKV_ERR_WORKSPACE;
    const long long rows = (long long)cache->num_blocks * cache->num_kv_heads * kBlockSize;
    // 16-bit tiles through tensor maps; INT8 tiles through tensor maps of the
    // codes (short-run kernel) or 1-D bulk copies (the 32-row kernel)
    CUtensorMap tk = {}, tv = {};
    if (pl.ops.src == kMqSrcMap &&
        (!encode_cache_map(&tk, k_cache, cache->kv_dtype == PKV_BF16, cache->head_dim, rows) ||
         !encode_cache_map(&tv, v_cache, cache->kv_dtype == PKV_BF16, cache->head_dim, rows)))
        return PKV_ERR_CUDA;
    MqI8Map mk = {}, mv = {};
    if (pl.ops.src == kMqSrcI8Map) {
        if (!encode_i8_map(&mk.map, k_cache, rows) || !encode_i8_map(&mv.map, v_cache, rows))
            return PKV_ERR_CUDA;
        mk.scales = k_scales;
        mv.scales = v_scales;
    }
    // Query runs of 16-bit caches that fill 128-row tiles take the tcgen05
    // kernel (no split, no combine, no workspace); shorter runs, and every run
    // over an INT8 cache, the mma.sync kernel below.
    // (With a window: where it pays, INT8 too, the wide-chunk kernel.)
    const bool wide = mq_aligned(q, 16) && mq_aligned(out, 16);
    const TcLaunch tc = wide && !win ? tc_for(cache, max_q_len, pl.G) : nullptr;
    const WideLaunch tw = wide && win ? wide_for(cache, q_dtype, batch, max_q_len, pl.G, max_blocks_per_seq,
                                                 window, sinks)
                                      : nullptr;
    if (tc || tw) {
        MqParams p;
        p.q = q; p.cu_q = cu_q; p.block_tables = block_tables; p.context_lens = context_lens;
        p.out = out; p.part_o = nullptr; p.part_ml = nullptr; p.ws_prefix = nullptr;
        p.status = dev_status;
        p.batch = batch; p.hq = num_q_heads; p.hkv = cache->num_kv_heads;
        p.mb = max_blocks_per_seq; p.num_blocks = cache->num_blocks; p.workers = 0;
        p.tmax = int(((long long)max_q_len * pl.G + kTcRows - 1) / kTcRows);
        p.max_q = max_q_len;
        p.qscale = softmax_scale * kMqLog2e;
        p.wait_ns = wait_ns < kTcWaitNs ? wait_ns : kTcWaitNs;
        p.stall_cta = stall_cta;
        p.window = window; p.sinks = sinks;
        const long long grid = (long long)batch * p.hkv * p.tmax;
        if (grid > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
        if (tw) {
            const MqI8Src ik{k_cache, k_scales}, iv{v_cache, v_scales};
            const void *ks = i8 ? static_cast<const void*>(&ik) : &tk, *vs = i8 ? static_cast<const void*>(&iv) : &tv;
            const long long pairs = (long long)batch * p.hkv * ((p.tmax + 1) / 2);
            if (tw(ks, vs, p, int(pairs), stream) != cudaSuccess) return PKV_ERR_CUDA;
        } else if (tc(tk, tv, p, int(grid), stream) != cudaSuccess) {
            return PKV_ERR_CUDA;
        }
        return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
    }
    char* ws = static_cast<char*>(workspace);
    MqParams p;
    p.q = q; p.cu_q = cu_q; p.block_tables = block_tables; p.context_lens = context_lens;
    p.out = out;
    p.part_o = reinterpret_cast<float*>(ws + pl.ws_o);
    p.part_ml = reinterpret_cast<float*>(ws + pl.ws_ml);
    p.ws_prefix = reinterpret_cast<int32_t*>(ws + pl.ws_prefix);
    p.status = dev_status;
    p.batch = batch; p.hq = num_q_heads; p.hkv = cache->num_kv_heads; p.mb = max_blocks_per_seq;
    p.num_blocks = cache->num_blocks; p.workers = int(pl.workers); p.tmax = pl.tmax;
    p.max_q = max_q_len;
    p.qscale = softmax_scale * kMqLog2e;
    p.wait_ns = wait_ns;
    p.stall_cta = stall_cta;
    p.window = window; p.sinks = sinks;
    if (pl.ops.prepare() != cudaSuccess) return PKV_ERR_CUDA;
    const MqI8Src ik{k_cache, k_scales}, iv{v_cache, v_scales};
    const void* ks = pl.ops.src == kMqSrcRaw ? static_cast<const void*>(&ik)
                     : pl.ops.src == kMqSrcI8Map ? static_cast<const void*>(&mk)
                                                 : static_cast<const void*>(&tk);
    const void* vs = pl.ops.src == kMqSrcRaw ? static_cast<const void*>(&iv)
                     : pl.ops.src == kMqSrcI8Map ? static_cast<const void*>(&mv)
                                                 : static_cast<const void*>(&tv);
    const long long ctas = (pl.workers + pl.ops.wpc - 1) / pl.ops.wpc;
    if (pl.ops.split(ks, vs, p, int(ctas), pl.smem, stream) != cudaSuccess)
        return PKV_ERR_CUDA;
    MqCombine cb;
    cb.part_o = p.part_o; cb.part_ml = p.part_ml; cb.ws_prefix = p.ws_prefix; cb.cu_q = cu_q;
    cb.context_lens = context_lens; cb.out = out; cb.batch = batch; cb.hq = num_q_heads;
    cb.hkv = p.hkv; cb.mb = max_blocks_per_seq; cb.workers = p.workers; cb.tmax = pl.tmax;
    cb.max_q = max_q_len; cb.window = window; cb.sinks = sinks;
    const long long grid = (long long)batch * p.hkv * pl.tmax;
    if (grid > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
    if (pl.ops.combine(cb, int(grid), stream) != cudaSuccess) return PKV_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

extern "C" pkv_status pkv_multiquery_attn(const void* q, pkv_dtype q_dtype, const int32_t* cu_q,
                                          int32_t max_q_len, const void* k_cache,
                                          const void* v_cache, const float* k_scales,
                                          const float* v_scales, const pkv_cache_desc* cache,
                                          const int32_t* block_tables, int32_t max_blocks_per_seq,
                                          const int32_t* context_lens, int32_t batch,
                                          int32_t num_q_heads, float softmax_scale, void* out,
                                          void* workspace, size_t workspace_bytes,
                                          int32_t num_parts, uint32_t* dev_status,
                                          cudaStream_t stream) {
    return run_multiquery(q, q_dtype, cu_q, max_q_len, k_cache, v_cache, k_scales, v_scales,
                          cache, block_tables, max_blocks_per_seq, context_lens, batch,
                          num_q_heads, softmax_scale, out, workspace, workspace_bytes, num_parts,
                          dev_status, stream, kMqWaitNs, -1);
}

extern "C" pkv_status pkv_window_multiquery_attn(
    const void* q, pkv_dtype q_dtype, const int32_t* cu_q, int32_t max_q_len, const void* k_cache,
    const void* v_cache, const float* k_scales, const float* v_scales, const pkv_cache_desc* cache,
    const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
    int32_t batch, int32_t num_q_heads, float softmax_scale, int32_t window, int32_t num_sinks,
    void* out, void* workspace, size_t workspace_bytes, int32_t num_parts, uint32_t* dev_status,
    cudaStream_t stream) {
    if (window < 0 || num_sinks < 0) return PKV_ERR_INVALID_ARG;
    return run_multiquery(q, q_dtype, cu_q, max_q_len, k_cache, v_cache, k_scales, v_scales,
                          cache, block_tables, max_blocks_per_seq, context_lens, batch,
                          num_q_heads, softmax_scale, out, workspace, workspace_bytes, num_parts,
                          dev_status, stream, kMqWaitNs, -1, true, window, num_sinks);
}

// ------------------------------------------------------------- test hook ---
#include "../../include/pkv_testing.h"

extern "C" pkv_status pkv_testing_window_multiquery_attn_stall(
    const void* q, pkv_dtype q_dtype, const int32_t* cu_q, int32_t max_q_len, const void* k_cache,
    const void* v_cache, const float* k_scales, const float* v_scales, const pkv_cache_desc* cache,
    const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
    int32_t batch, int32_t num_q_heads, float softmax_scale, int32_t window, int32_t num_sinks,
    void* out, void* workspace, size_t workspace_bytes, int32_t num_parts, uint64_t wait_limit_ns,
    int32_t stall_cta, uint32_t* dev_status, cudaStream_t stream) {
    if (window < 0 || num_sinks < 0 || wait_limit_ns > kMqWaitNs || stall_cta < -1)
        return PKV_ERR_INVALID_ARG;
    return run_multiquery(q, q_dtype, cu_q, max_q_len, k_cache, v_cache, k_scales, v_scales,
                          cache, block_tables, max_blocks_per_seq, context_lens, batch,
                          num_q_heads, softmax_scale, out, workspace, workspace_bytes, num_parts,
                          dev_status, stream, wait_limit_ns, stall_cta, true, window, num_sinks);
}

static void planned_split(const MqPlan& pl, int32_t* kernel, int32_t* rows_per_tile) {
    *kernel = pl.ops.src == kMqSrcI8Map ? PKV_TESTING_MQ_SHORT_I8
              : pl.ops.wpc > 1          ? PKV_TESTING_MQ_SHORT
                                        : PKV_TESTING_MQ_ROWS16;
    *rows_per_tile = pl.ops.rt;
}

extern "C" pkv_status pkv_testing_window_multiquery_kernel(
    int32_t batch, int32_t num_q_heads, int32_t max_q_len, const pkv_cache_desc* cache,
    pkv_dtype q_dtype, int32_t max_blocks_per_seq, int32_t window, int32_t num_sinks,
    int32_t num_parts, int32_t* kernel, int32_t* rows_per_tile) {
    if (!kernel || !rows_per_tile || num_parts <= 0 || max_blocks_per_seq <= 0 || window < 0 ||
        num_sinks < 0)
        return PKV_ERR_INVALID_ARG;
    MqPlan pl;
    const pkv_status s = mq_plan(cache, batch, num_q_heads, max_q_len, q_dtype, num_parts, &pl, true);
    if (s != PKV_OK) return s;
    if (wide_for(cache, q_dtype, batch, max_q_len, pl.G, max_blocks_per_seq, window, num_sinks)) {
        *kernel = PKV_TESTING_MQ_WIDE;
        *rows_per_tile = kTcRows;
        return PKV_OK;
    }
    planned_split(pl, kernel, rows_per_tile);
    return PKV_OK;
}

extern "C" pkv_status pkv_testing_multiquery_kernel(int32_t batch, int32_t num_q_heads,
                                                    int32_t max_q_len, const pkv_cache_desc* cache,
                                                    pkv_dtype q_dtype, int32_t num_parts,
                                                    int32_t* kernel, int32_t* rows_per_tile) {
    if (!kernel || !rows_per_tile || num_parts <= 0) return PKV_ERR_INVALID_ARG;
    MqPlan pl;
    const pkv_status s = mq_plan(cache, batch, num_q_heads, max_q_len, q_dtype, num_parts, &pl);
    if (s != PKV_OK) return s;
    if (tc_for(cache, max_q_len, pl.G)) {
        *kernel = PKV_TESTING_MQ_TCGEN05;
        *rows_per_tile = kTcRows;
        return PKV_OK;
    }
    planned_split(pl, kernel, rows_per_tile);
    return PKV_OK;
}

extern "C" pkv_status pkv_testing_multiquery_attn_stall(
    const void* q, pkv_dtype q_dtype, const int32_t* cu_q, int32_t max_q_len, const void* k_cache,
    const void* v_cache, const float* k_scales, const float* v_scales,
    const pkv_cache_desc* cache, const int32_t* block_tables,
    int32_t max_blocks_per_seq, const int32_t* context_lens, int32_t batch, int32_t num_q_heads,
    float softmax_scale, void* out, void* workspace, size_t workspace_bytes, int32_t num_parts,
    uint64_t wait_limit_ns, int32_t stall_cta, uint32_t* dev_status, cudaStream_t stream) {
    if (wait_limit_ns > kMqWaitNs || stall_cta < -1) return PKV_ERR_INVALID_ARG;
    return run_multiquery(q, q_dtype, cu_q, max_q_len, k_cache, v_cache, k_scales, v_scales,
                          cache, block_tables, max_blocks_per_seq, context_lens, batch,
                          num_q_heads, softmax_scale, out, workspace, workspace_bytes, num_parts,
                          dev_status, stream, wait_limit_ns, stall_cta);
}
