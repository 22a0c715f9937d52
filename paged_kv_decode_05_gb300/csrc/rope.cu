// Norms of queries and keys for each head, the position rotation, and the
// write of K and V into the paged cache, in one pass.
//
// For a head row x of D values: y_d = x_d r w_d with r = rsqrt(mean_d x_d^2 +
// eps) (without weights y = x), then the pairs (u, v) of the first rot_dim
// values turn by their token's angle, (u c - v s, u s + v c), c and s from a
// table row of the pair's position axis. All in fp32, rounded once to the
// 16-bit type. Bound by memory: every row is read and written once, and a
// token's table rows are read once per warp, which keeps them in registers
// for all the head rows that it handles.
//
// A row takes D / 8 lanes of two 8-byte parts each, so a warp handles 2 (D =
// 128) or 4 (D = 64) rows side by side. The parts are chosen so that a lane
// holds both values of its pairs: values [4c, 4c + 4) and their partners half a
// rotation further on, or 8 consecutive values if pairs are interleaved. (With
// 16 consecutive bytes per lane the partners came from another lane: 8 shuffles
// and 8 selects more per row, 50 M instead of XX M instructions and 71 instead
// of XX us on 8191 tokens of 48 heads of 128.)
#include "common.cuh"

namespace pkv {
namespace {

constexpr int kMaxPairs = 64;

struct RopeParams {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;              // append only
    long long q_stride, k_stride, v_stride;   // elements between tokens
    const uint16_t* q_weight;       // [D] or nullptr
    const uint16_t* k_weight;
    const float* cos_sin;           // [max_position, rot]: cos of the pairs, then sin
    const int32_t* positions;       // [axes, tokens]
    const int64_t* slots;           // append only
    uint16_t* q_out;                // [tokens, hq, D]
    uint16_t* k_out;                // [tokens, hkv, D], or the K cache
    uint16_t* v_out;                // append only: the V cache
    uint32_t* status;
    long long pool_slots;
    float eps;
    int tokens, hq, hkv, rot, max_position, axes;
    int gq, gk, groups;             // row groups of q, of k, and all (v last) of a token
    int chunks, per_chunk;          // warps per token, row groups per warp
    unsigned char axis[kMaxPairs];
};

__device__ __forceinline__ float4 unpack4(BF16 t, const uint2& w) {
    const float2 a = unpack2(t, w.x), b = unpack2(t, w.y);
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float4 unpack4(F16 t, const uint2& w) {
    const float2 a = unpack2(t, w.x), b = unpack2(t, w.y);
    return make_float4(a.x, a.y, b.x, b.y);
}

template <typename T, int D, bool APPEND, bool INTER>
__global__ void __launch_bounds__(128) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;      // lanes per row, rows per warp
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, col = lane % LPR, sub = lane / LPR;
    const long long task = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (task >= (long long)p.tokens * p.chunks) return;
    const int n = int(task / p.chunks), chunk = int(task - (long long)n * p.chunks);

    // this lane's values: da + [0, 4) and db + [0, 4)
    const int half = p.rot / 2;
    const bool turns = INTER ? 8 * col < p.rot : 4 * col < half;
    const int da = INTER ? 8 * col : (turns ? 4 * col : p.rot + 8 * (col - half / 4));
    const int db = INTER || !turns ? da + 4 : da + half;

    // a row group: its source and destination rows (nullptr: nothing there)
    long long cache_row = -1;     // append: (block hkv) * 16 + row of kv head 0
    auto source = [&](int g) -> const uint16_t* {
        if (g < p.gq) {
            const int r = g * RPW + sub;
            return r < p.hq ? p.q + n * p.q_stride + r * D : nullptr;
        }
        const bool is_k = g < p.gq + p.gk;
        const int r = (g - p.gq - (is_k ? 0 : p.gk)) * RPW + sub;
        if (r >= p.hkv) return nullptr;
        return (is_k ? p.k + n * p.k_stride : p.v + n * p.v_stride) + r * D;
    };
    auto target = [&](int g) -> uint16_t* {
        if (g < p.gq) return p.q_out + ((long long)n * p.hq + g * RPW + sub) * D;
        const bool is_k = g < p.gq + p.gk;
        const int r = (g - p.gq - (is_k ? 0 : p.gk)) * RPW + sub;
        if constexpr (APPEND) {
            if (cache_row < 0) return nullptr;
            return (is_k ? p.k_out : p.v_out) + (cache_row + (long long)r * kBlockSize) * D;
        } else {
            return p.k_out + ((long long)n * p.hkv + r) * D;
        }
    };
    auto load = [&](const uint16_t* src, uint2& a, uint2& b) {
        a = b = make_uint2(0u, 0u);
        if (src == nullptr) return;
        a = *reinterpret_cast<const uint2*>(src + da);
        b = *reinterpret_cast<const uint2*>(src + db);
    };
    const int g0 = chunk * p.per_chunk, g1 = min(p.groups, g0 + p.per_chunk);
    const uint16_t* src = source(g0);
    uint2 ra, rb;
    load(src, ra, rb);            // the first rows travel while the angles are looked up

    bool bad = false;
    for (int a = 0; a < p.axes; ++a)
        bad |= unsigned(p.positions[(long long)a * p.tokens + n]) >= unsigned(p.max_position);
    if (bad) {
        if (chunk == 0 && lane == 0) flag_status(p.status, PKV_DEV_BAD_INDEX);
        return;
    }
    float cs[4], sn[4];
    if (turns) {
        const int j0 = 4 * col, a = p.axis[j0];
        if (p.axis[j0 + 1] == a && p.axis[j0 + 2] == a && p.axis[j0 + 3] == a) {
            const float* r = p.cos_sin + (long long)p.positions[(long long)a * p.tokens + n] * p.rot + j0;
            const float4 c = __ldg(reinterpret_cast<const float4*>(r));
            const float4 s = __ldg(reinterpret_cast<const float4*>(r + half));
            cs[0] = c.x; cs[1] = c.y; cs[2] = c.z; cs[3] = c.w;
            sn[0] = s.x; sn[1] = s.y; sn[2] = s.z; sn[3] = s.w;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int ak = p.axis[j0 + k];
                const float* r = p.cos_sin + (long long)p.positions[(long long)ak * p.tokens + n] * p.rot + j0 + k;
                cs[k] = __ldg(r);
                sn[k] = __ldg(r + half);
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) { cs[k] = 1.f; sn[k] = 0.f; }
    }
    if constexpr (APPEND) {
        const long long slot = p.slots[n];
        if (slot >= p.pool_slots) {
            if (chunk == 0 && lane == 0) flag_status(p.status, PKV_DEV_BAD_SLOT);
        } else if (slot >= 0) {
            cache_row = (slot / kBlockSize) * p.hkv * kBlockSize + slot % kBlockSize;
        }
    }

    float4 wa, wb;                // weights of the current kind of row
    const uint16_t* w = nullptr;
    for (int g = g0; g < g1; ++g) {
        uint2 xa = ra, xb = rb;
        const bool in = src != nullptr;
        if (g + 1 < g1) {         // the next rows travel while these are worked on
            src = source(g + 1);
            load(src, ra, rb);
        }
        if (g < p.gq + p.gk) {
            if (g == g0 || g == p.gq) {
                w = g < p.gq ? p.q_weight : p.k_weight;
                if (w != nullptr) {
                    wa = unpack4(T{}, __ldg(reinterpret_cast<const uint2*>(w + da)));
                    wb = unpack4(T{}, __ldg(reinterpret_cast<const uint2*>(w + db)));
                }
            }
            float4 a = unpack4(T{}, xa), b = unpack4(T{}, xb);
            if (w != nullptr) {
                float ss = a.x * a.x + a.y * a.y + a.z * a.z + a.w * a.w + b.x * b.x + b.y * b.y +
                           b.z * b.z + b.w * b.w;
#pragma unroll
                for (int off = 1; off < LPR; off <<= 1) ss += __shfl_xor_sync(kFull, ss, off);
                const float rn = rsqrtf(ss * (1.f / D) + p.eps);
                a.x *= rn * wa.x; a.y *= rn * wa.y; a.z *= rn * wa.z; a.w *= rn * wa.w;
                b.x *= rn * wb.x; b.y *= rn * wb.y; b.z *= rn * wb.z; b.w *= rn * wb.w;
            }
            float4 ya, yb;
            if constexpr (INTER) {
                ya = make_float4(a.x * cs[0] - a.y * sn[0], a.x * sn[0] + a.y * cs[0],
                                 a.z * cs[1] - a.w * sn[1], a.z * sn[1] + a.w * cs[1]);
                yb = make_float4(b.x * cs[2] - b.y * sn[2], b.x * sn[2] + b.y * cs[2],
                                 b.z * cs[3] - b.w * sn[3], b.z * sn[3] + b.w * cs[3]);
            } else {
                ya = make_float4(a.x * cs[0] - b.x * sn[0], a.y * cs[1] - b.y * sn[1],
                                 a.z * cs[2] - b.z * sn[2], a.w * cs[3] - b.w * sn[3]);
                yb = make_float4(a.x * sn[0] + b.x * cs[0], a.y * sn[1] + b.y * cs[1],
                                 a.z * sn[2] + b.z * cs[2], a.w * sn[3] + b.w * cs[3]);
            }
            if (!turns) { ya = a; yb = b; }      // also where 0 * inf would make NaN
            xa = make_uint2(pack2<T>(ya.x, ya.y), pack2<T>(ya.z, ya.w));
            xb = make_uint2(pack2<T>(yb.x, yb.y), pack2<T>(yb.z, yb.w));
        }                         // v rows are copied bit for bit
        uint16_t* dst = in ? target(g) : nullptr;
        if (dst != nullptr) {
            *reinterpret_cast<uint2*>(dst + da) = xa;
            *reinterpret_cast<uint2*>(dst + db) = xb;
        }
    }
}

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <typename T, int D, bool APPEND>
cudaError_t launch_rope(const RopeParams& p, bool inter, cudaStream_t st) {
    const long long tasks = (long long)p.tokens * p.chunks;
    const dim3 grid(unsigned((tasks + 3) / 4)), block(128);
    return inter ? launch_pdl(qk_norm_rope_kernel<T, D, APPEND, true>, grid, block, 0, st, p)
                 : launch_pdl(qk_norm_rope_kernel<T, D, APPEND, false>, grid, block, 0, st, p);
}

struct RopeArgs {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    pkv_dtype dtype;
    int32_t tokens, hq, hkv, head_dim;
    const void *q_weight, *k_weight;
    float eps;
    const float* cos_sin;
    int32_t max_position, rot_dim, interleaved;
    const int32_t* positions;
    int32_t axes;
    const int32_t* pair_axis;      // host
    void *q_out, *k_out, *v_out;
    const int64_t* slots;
    long long pool_slots;
    uint32_t* status;
};

template <bool APPEND>
pkv_status run_rope(const RopeArgs& a, cudaStream_t st) {
    if (a.dtype != PKV_F16 && a.dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
    if (a.tokens < 0 || a.hq <= 0 || a.hkv <= 0 || a.hq > 0xffff || a.hkv > 0xffff)
        return PKV_ERR_INVALID_ARG;
    if (a.head_dim != 64 && a.head_dim != 128) return PKV_ERR_UNSUPPORTED;
    const int D = a.head_dim;
    if (a.rot_dim < 0 || a.rot_dim > D || (a.interleaved != 0 && a.interleaved != 1))
        return PKV_ERR_INVALID_ARG;
    if (a.rot_dim % 16 != 0) return PKV_ERR_UNSUPPORTED;
    if (!(a.eps >= 0.f && a.eps <= 3.0e38f)) return PKV_ERR_INVALID_ARG;
    const long long row_q = (long long)a.hq * D, row_k = (long long)a.hkv * D;
    if (a.q_stride < row_q || a.k_stride < row_k || (APPEND && a.v_stride < row_k) ||
        a.q_stride % 8 || a.k_stride % 8 || (APPEND && a.v_stride % 8))
        return PKV_ERR_INVALID_ARG;
    if (a.rot_dim > 0) {
        if (a.axes < 1 || a.axes > 4 || a.max_position <= 0) return PKV_ERR_INVALID_ARG;
        for (int j = 0; a.pair_axis && j < a.rot_dim / 2; ++j)
            if (a.pair_axis[j] < 0 || a.pair_axis[j] >= a.axes) return PKV_ERR_INVALID_ARG;
    }
    if (a.tokens == 0) return PKV_OK;
    if (!a.q || !a.k || !a.q_out || !a.k_out) return PKV_ERR_INVALID_ARG;
    if (APPEND && (!a.v || !a.v_out || !a.slots)) return PKV_ERR_INVALID_ARG;
    if (a.rot_dim > 0 && (!a.cos_sin || !a.positions)) return PKV_ERR_INVALID_ARG;
    if (!aligned_to(a.q, 16) || !aligned_to(a.k, 16) || !aligned_to(a.v, 16) ||
        !aligned_to(a.q_out, 16) || !aligned_to(a.k_out, 16) || !aligned_to(a.v_out, 16) ||
        !aligned_to(a.q_weight, 16) || !aligned_to(a.k_weight, 16) || !aligned_to(a.cos_sin, 16) ||
        !aligned_to(a.positions, 4) || !aligned_to(a.slots, 8) || !aligned_to(a.status, 4))
        return PKV_ERR_INVALID_ARG;
    // in place: a warp reads a row before it writes it, but rows must coincide
    if ((a.q_out == a.q && a.q_stride != row_q) || (!APPEND && a.k_out == a.k && a.k_stride != row_k))
        return PKV_ERR_INVALID_ARG;

    RopeParams p;
    p.q = static_cast<const uint16_t*>(a.q);
    p.k = static_cast<const uint16_t*>(a.k);
    p.v = static_cast<const uint16_t*>(a.v);
    p.q_stride = a.q_stride; p.k_stride = a.k_stride; p.v_stride = a.v_stride;
    p.q_weight = static_cast<const uint16_t*>(a.q_weight);
    p.k_weight = static_cast<const uint16_t*>(a.k_weight);
    p.cos_sin = a.cos_sin; p.positions = a.positions; p.slots = a.slots;
    p.q_out = static_cast<uint16_t*>(a.q_out);
    p.k_out = static_cast<uint16_t*>(a.k_out);
    p.v_out = static_cast<uint16_t*>(a.v_out);
    p.status = a.status; p.pool_slots = a.pool_slots; p.eps = a.eps;
    p.tokens = a.tokens; p.hq = a.hq; p.hkv = a.hkv; p.rot = a.rot_dim;
    p.max_position = a.max_position;
    p.axes = a.rot_dim > 0 ? a.axes : 0;
    for (int j = 0; j < kMaxPairs; ++j)
        p.axis[j] = (unsigned char)(a.pair_axis && j < a.rot_dim / 2 ? a.pair_axis[j] : 0);
    // One row group per warp while that fills the device; with more tokens a
    // warp keeps its angles for up to 8 groups.
    const int rpw = 32 * 8 / D;
    p.gq = (a.hq + rpw - 1) / rpw;
    p.gk = (a.hkv + rpw - 1) / rpw;
    p.groups = p.gq + (APPEND ? 2 : 1) * p.gk;
    long long per = (long long)a.tokens * p.groups / (152 * 32);
    per = per < 1 ? 1 : (per > 8 ? 8 : per);
    p.per_chunk = int(per);
    p.chunks = (p.groups + p.per_chunk - 1) / p.per_chunk;
    if (((long long)a.tokens * p.chunks + 3) / 4 > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
    const bool inter = a.interleaved != 0;
    cudaError_t e;
    if (a.dtype == PKV_BF16)
        e = D == 128 ? launch_rope<BF16, 128, APPEND>(p, inter, st) : launch_rope<BF16, 64, APPEND>(p, inter, st);
    else
        e = D == 128 ? launch_rope<F16, 128, APPEND>(p, inter, st) : launch_rope<F16, 64, APPEND>(p, inter, st);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_qk_norm_rope(
    const void* q, int64_t q_stride, const void* k, int64_t k_stride, pkv_dtype dtype,
    int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
    const void* q_weight, const void* k_weight, float eps, const float* cos_sin,
    int32_t max_position, int32_t rot_dim, int32_t interleaved, const int32_t* positions,
    int32_t num_axes, const int32_t* pair_axis, void* q_out, void* k_out, uint32_t* dev_status,
    cudaStream_t stream) {
    RopeArgs a = {};
    a.q = q; a.k = k; a.q_stride = q_stride; a.k_stride = k_stride;
    a.dtype = dtype; a.tokens = num_tokens; a.hq = num_q_heads; a.hkv = num_kv_heads;
    a.head_dim = head_dim; a.q_weight = q_weight; a.k_weight = k_weight; a.eps = eps;
    a.cos_sin = cos_sin; a.max_position = max_position; a.rot_dim = rot_dim;
    a.interleaved = interleaved; a.positions = positions; a.axes = num_axes; a.pair_axis = pair_axis;
    a.q_out = q_out; a.k_out = k_out; a.status = dev_status;
    return run_rope<false>(a, stream);
}

extern "C" pkv_status pkv_qk_norm_rope_append(
    const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
    int64_t v_stride, pkv_dtype dtype, int32_t num_tokens, int32_t num_q_heads,
    const void* q_weight, const void* k_weight, float eps, const float* cos_sin,
    int32_t max_position, int32_t rot_dim, int32_t interleaved, const int32_t* positions,
    int32_t num_axes, const int32_t* pair_axis, void* q_out, const int64_t* slot_mapping,
    void* k_cache, void* v_cache, const pkv_cache_desc* cache, uint32_t* dev_status,
    cudaStream_t stream) {
    if (!cache || cache->num_blocks <= 0 || cache->num_kv_heads <= 0) return PKV_ERR_INVALID_ARG;
    if (cache->kv_dtype != PKV_F16 && cache->kv_dtype != PKV_BF16 && cache->kv_dtype != PKV_I8)
        return PKV_ERR_INVALID_ARG;
    if (cache->block_size != kBlockSize || cache->kv_dtype == PKV_I8) return PKV_ERR_UNSUPPORTED;
    if (dtype != cache->kv_dtype) return PKV_ERR_INVALID_ARG;
    RopeArgs a = {};
    a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.dtype = dtype; a.tokens = num_tokens; a.hq = num_q_heads; a.hkv = cache->num_kv_heads;
    a.head_dim = cache->head_dim; a.q_weight = q_weight; a.k_weight = k_weight; a.eps = eps;
    a.cos_sin = cos_sin; a.max_position = max_position; a.rot_dim = rot_dim;
    a.interleaved = interleaved; a.positions = positions; a.axes = num_axes; a.pair_axis = pair_axis;
    a.q_out = q_out; a.k_out = k_cache; a.v_out = v_cache; a.slots = slot_mapping;
    a.pool_slots = (long long)cache->num_blocks * kBlockSize; a.status = dev_status;
    return run_rope<true>(a, stream);
}
