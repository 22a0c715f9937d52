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
// A row takes D / 8 lanes of 16 bytes each, so a warp handles 2 (D = 128) or
// 4 (D = 64) rows side by side; the other half of a pair is in another lane of
// the row (halves) or in the same one (interleaved).
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
    int rows, chunks, per_chunk;    // head rows of a token, its warps, row groups per warp
    unsigned char axis[kMaxPairs];
};

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
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

    // the token's angles for this lane's 8 values
    const int half = p.rot / 2, d0 = 8 * col;
    constexpr int NP = INTER ? 4 : 8;
    float cs[NP], sn[NP];
    const bool turns = d0 < p.rot;
    bool bad = false;
    for (int a = 0; a < p.axes; ++a) {
        const int x = p.positions[(long long)a * p.tokens + n];
        bad |= unsigned(x) >= unsigned(p.max_position);
    }
    if (bad) {
        if (chunk == 0 && lane == 0) flag_status(p.status, PKV_DEV_BAD_INDEX);
        return;
    }
    if (turns) {
        const int j0 = INTER ? d0 / 2 : (d0 < half ? d0 : d0 - half);
#pragma unroll
        for (int i = 0; i < NP; i += 4) {
            const int a = p.axis[j0 + i];
            if (p.axis[j0 + i + 1] == a && p.axis[j0 + i + 2] == a && p.axis[j0 + i + 3] == a) {
                const float* r = p.cos_sin + (long long)p.positions[(long long)a * p.tokens + n] * p.rot + j0 + i;
                const float4 c = __ldg(reinterpret_cast<const float4*>(r));
                const float4 s = __ldg(reinterpret_cast<const float4*>(r + half));
                cs[i] = c.x; cs[i + 1] = c.y; cs[i + 2] = c.z; cs[i + 3] = c.w;
                sn[i] = s.x; sn[i + 1] = s.y; sn[i + 2] = s.z; sn[i + 3] = s.w;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int ak = p.axis[j0 + i + k];
                    const float* r = p.cos_sin + (long long)p.positions[(long long)ak * p.tokens + n] * p.rot + j0 + i + k;
                    cs[i + k] = __ldg(r);
                    sn[i + k] = __ldg(r + half);
                }
            }
        }
    }
    // the lane that holds the other values of this lane's pairs
    const int shift = half / 8;
    const int other = INTER || !turns ? lane : (d0 < half ? lane + shift : lane - shift);

    long long cache_row = -1;     // append: (block hkv) * 16 + row of kv head 0
    if constexpr (APPEND) {
        const long long slot = p.slots[n];
        if (slot >= p.pool_slots) {
            if (chunk == 0 && lane == 0) flag_status(p.status, PKV_DEV_BAD_SLOT);
        } else if (slot >= 0) {
            cache_row = (slot / kBlockSize) * p.hkv * kBlockSize + slot % kBlockSize;
        }
    }

    const int g0 = chunk * p.per_chunk;
    for (int g = g0; g < g0 + p.per_chunk; ++g) {
        const int r = g * RPW + sub;
        if (g * RPW >= p.rows) break;
        const bool in = r < p.rows, is_q = r < p.hq, is_k = !is_q && r < p.hq + p.hkv;
        const uint16_t* src = nullptr;
        uint16_t* dst = nullptr;
        if (in) {
            if (is_q) {
                src = p.q + n * p.q_stride + r * D;
                dst = p.q_out + ((long long)n * p.hq + r) * D;
            } else {
                const int h = is_k ? r - p.hq : r - p.hq - p.hkv;
                src = (is_k ? p.k + n * p.k_stride : p.v + n * p.v_stride) + h * D;
                if constexpr (APPEND) {
                    if (cache_row >= 0)
                        dst = (is_k ? p.k_out : p.v_out) + (cache_row + (long long)h * kBlockSize) * D;
                } else {
                    dst = p.k_out + ((long long)n * p.hkv + h) * D;
                }
            }
        }
        uint4 raw = make_uint4(0u, 0u, 0u, 0u);
        if (in) raw = *reinterpret_cast<const uint4*>(src + d0);
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2(T{}, word(raw, i));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
        const uint16_t* w = is_q ? p.q_weight : is_k ? p.k_weight : nullptr;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int off = 1; off < LPR; off <<= 1) ss += __shfl_xor_sync(kFull, ss, off);
        if (w != nullptr && in) {
            const float rn = rsqrtf(ss * (1.f / D) + p.eps);
            const uint4 ww = __ldg(reinterpret_cast<const uint4*>(w + d0));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack2(T{}, word(ww, i));
                x[2 * i] *= rn * f.x;
                x[2 * i + 1] *= rn * f.y;
            }
        }
        float y[8];
        if constexpr (INTER) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[2 * i] = x[2 * i];
                y[2 * i + 1] = x[2 * i + 1];
                if (turns) {
                    y[2 * i] = x[2 * i] * cs[i] - x[2 * i + 1] * sn[i];
                    y[2 * i + 1] = x[2 * i] * sn[i] + x[2 * i + 1] * cs[i];
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float o = __shfl_sync(kFull, x[i], other);
                y[i] = x[i];
                if (turns) y[i] = d0 < half ? x[i] * cs[i] - o * sn[i] : o * sn[i] + x[i] * cs[i];
            }
        }
        if (dst != nullptr) {
            uint4 res = raw;                                      // v rows are copied bit for bit
            if (is_q || is_k)
                res = make_uint4(pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3]), pack2<T>(y[4], y[5]),
                                 pack2<T>(y[6], y[7]));
            *reinterpret_cast<uint4*>(dst + d0) = res;
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
    p.rows = a.hq + (APPEND ? 2 : 1) * a.hkv;
    const int rpw = 32 * 8 / D, groups = (p.rows + rpw - 1) / rpw;
    long long per = (long long)a.tokens * groups / (152 * 32);
    per = per < 1 ? 1 : (per > 8 ? 8 : per);
    p.per_chunk = int(per);
    p.chunks = (groups + p.per_chunk - 1) / p.per_chunk;
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
