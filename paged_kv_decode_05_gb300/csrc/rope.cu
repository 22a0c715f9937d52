// Norms of queries and keys for each head, the position rotation, and the
// write of K and V into the paged cache, in one pass.
//
// For a head row x of D values: y_d = x_d r w_d with r = rsqrt(mean_d x_d^2 +
// eps) (without weights y = x), then the pairs (u, v) of the first rot_dim
// values turn by their token's angle, (u c - v s, u s + v c), c and s from a
// table row of the pair's position axis. All in fp32, rounded once to the
// 16-bit type. Bound by memory: every row is read and written once. 8191 tokens
// of 48 heads of 128, three axes: 38.4 us for 205 MB, 0.80 of the measured copy
// rate (a plain copy of the same bytes takes 31 us, 4 of the rest are the
// launch's ramp); 71 us as one loop over a token's rows with scalar arithmetic.
// One token: 2.2 us, a launch.
//
// A row takes D / 8 lanes of two 8-byte parts each, so a warp handles 2 (D =
// 128) or 4 (D = 64) rows side by side. The parts are chosen so that a lane
// holds both values of its pairs: values [4c, 4c + 4) and their partners half a
// rotation further on, or 8 consecutive values if pairs are interleaved: no
// shuffles but for the sum of squares. The arithmetic is in packed fp32 pairs
// (fma.rn.f32x2), half the instructions of scalar code.
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
    int cq, ck, chunks;             // warps of q, of k, and all (v last) of a token
    int per_chunk;                  // row groups per warp
    int stride;                     // tokens that are worked on side by side
    alignas(4) unsigned char axis[kMaxPairs];
};

// Two fp32 values in one 64-bit register pair, and the packed instructions.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 split(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
template <typename T>
__device__ __forceinline__ f32x2 load2(uint32_t w) {
    const float2 f = unpack2(T{}, w);
    return pair(f.x, f.y);
}
template <typename T>
__device__ __forceinline__ uint32_t store2(f32x2 v) {
    const float2 f = split(v);
    return pack2<T>(f.x, f.y);
}

constexpr int kGroups = 4;        // row groups of a warp, at most

// A warp takes one kind of row (q, k or v), up to kGroups row groups of it, and
// every stride-th token. A token's position and slot are asked for one token
// ahead, so that its rows and its angles travel together and a warp waits for
// memory once per token.
template <typename T, int D, bool APPEND, bool INTER>
__global__ void __launch_bounds__(128, 8) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;      // lanes per row, rows per warp
    constexpr int U = kGroups;
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, col = lane % LPR, sub = lane / LPR;
    const int wid = int(blockIdx.x) * 4 + int(threadIdx.x >> 5);
    int n = wid / p.chunks, chunk = wid - n * p.chunks;
    if (n >= p.stride) return;
    const bool first = chunk == 0;
    // kind of row: 0 q, 1 k, 2 v
    const int kind = chunk < p.cq ? 0 : (chunk < p.cq + p.ck ? 1 : 2);
    chunk -= kind == 0 ? 0 : (kind == 1 ? p.cq : p.cq + p.ck);
    const int row0 = chunk * p.per_chunk * RPW + sub;
    const int rows = min(kind == 0 ? p.hq : p.hkv, (chunk + 1) * p.per_chunk * RPW);
    const long long src_step = kind == 0 ? p.q_stride : kind == 1 ? p.k_stride : p.v_stride;
    const uint16_t* src0 = (kind == 0 ? p.q : kind == 1 ? p.k : p.v) + row0 * D;

    // this lane's values: da + [0, 4) and db + [0, 4)
    const int half = p.rot / 2;
    const bool turns = kind != 2 && (INTER ? 8 * col < p.rot : 4 * col < half);
    int da = 8 * col, db = 8 * col + 4;
    if (!INTER && kind != 2) {
        da = turns ? 4 * col : p.rot + 8 * (col - half / 4);
        db = turns ? da + half : da + 4;
    }
    const uint16_t* w = kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr;
    uint2 wa = make_uint2(0u, 0u), wb = wa;
    if (w != nullptr) {
        wa = __ldg(reinterpret_cast<const uint2*>(w + da));
        wb = __ldg(reinterpret_cast<const uint2*>(w + db));
    }
    const int j0 = turns ? 4 * col : 0;
    const uint32_t axis = *reinterpret_cast<const uint32_t*>(p.axis + j0);   // of 4 pairs
    const bool one_axis = axis == (axis & 0xff) * 0x01010101u;

    // lane a holds the position on axis a
    int at = lane < p.axes ? p.positions[(long long)lane * p.tokens + n] : 0;
    long long slot = APPEND ? p.slots[n] : 0;
    for (; n < p.tokens; n += p.stride) {
        const int at_n = at;
        const long long slot_n = slot;
        if (n < p.tokens - p.stride) {
            if (lane < p.axes) at = p.positions[(long long)lane * p.tokens + n + p.stride];
            if constexpr (APPEND) slot = p.slots[n + p.stride];
        }
        uint2 xa[U], xb[U];
        const uint16_t* src = src0 + n * src_step;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            xa[i] = xb[i] = make_uint2(0u, 0u);
            if (row0 + i * RPW < rows) {
                xa[i] = *reinterpret_cast<const uint2*>(src + i * (RPW * D) + da);
                xb[i] = *reinterpret_cast<const uint2*>(src + i * (RPW * D) + db);
            }
        }
        if (__any_sync(kFull, lane < p.axes && unsigned(at_n) >= unsigned(p.max_position))) {
            if (first && lane == 0) flag_status(p.status, PKV_DEV_BAD_INDEX);
            continue;
        }
        f32x2 cs[2], sn[2], ms[2];    // cos, sin, -sin of the lane's 4 pairs
        if (kind != 2 && p.rot > 0) { // warp-uniform
            float c[4], s[4];
            int pos[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) pos[k] = __shfl_sync(kFull, at_n, (axis >> (8 * k)) & 0xff);
            if (one_axis) {
                const float* r = p.cos_sin + (long long)pos[0] * p.rot + j0;
                const float4 cv = __ldg(reinterpret_cast<const float4*>(r));
                const float4 sv = __ldg(reinterpret_cast<const float4*>(r + half));
                c[0] = cv.x; c[1] = cv.y; c[2] = cv.z; c[3] = cv.w;
                s[0] = sv.x; s[1] = sv.y; s[2] = sv.z; s[3] = sv.w;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float* r = p.cos_sin + (long long)pos[k] * p.rot + j0 + k;
                    c[k] = __ldg(r);
                    s[k] = __ldg(r + half);
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                cs[i] = pair(c[2 * i], c[2 * i + 1]);
                sn[i] = pair(s[2 * i], s[2 * i + 1]);
                ms[i] = pair(-s[2 * i], -s[2 * i + 1]);
            }
        }

        uint16_t* dst;
        long long dst_row = D;        // elements between the rows of consecutive heads
        if (kind == 0) {
            dst = p.q_out + (long long)n * p.hq * D;
        } else if constexpr (APPEND) {
            if (slot_n >= p.pool_slots && kind == 1 && chunk == 0 && lane == 0)
                flag_status(p.status, PKV_DEV_BAD_SLOT);
            if (slot_n < 0 || slot_n >= p.pool_slots) continue;
            dst_row = kBlockSize * D;
            dst = (kind == 1 ? p.k_out : p.v_out) +
                  ((slot_n / kBlockSize) * p.hkv * kBlockSize + slot_n % kBlockSize) * D;
        } else {
            dst = p.k_out + (long long)n * p.hkv * D;
        }
        dst += row0 * dst_row;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (i >= p.per_chunk) break;
            if (kind != 2) {          // v rows are copied bit for bit
                f32x2 a0 = load2<T>(xa[i].x), a1 = load2<T>(xa[i].y);
                f32x2 b0 = load2<T>(xb[i].x), b1 = load2<T>(xb[i].y);
                if (w != nullptr) {
                    const float2 s2 = split(fma2(b1, b1, fma2(b0, b0, fma2(a1, a1, mul2(a0, a0)))));
                    float ss = s2.x + s2.y;
#pragma unroll
                    for (int off = 1; off < LPR; off <<= 1) ss += __shfl_xor_sync(kFull, ss, off);
                    const float r = rsqrtf(ss * (1.f / D) + p.eps);
                    const f32x2 rr = pair(r, r);
                    a0 = mul2(a0, mul2(rr, load2<T>(wa.x)));
                    a1 = mul2(a1, mul2(rr, load2<T>(wa.y)));
                    b0 = mul2(b0, mul2(rr, load2<T>(wb.x)));
                    b1 = mul2(b1, mul2(rr, load2<T>(wb.y)));
                }
                if (turns) {
                    if constexpr (INTER) {
                        // pairs (a0.x, a0.y), (a1.x, a1.y), (b0.x, b0.y), (b1.x, b1.y)
                        auto turn = [](f32x2& v, float c, float s) {
                            const float2 x = split(v);
                            v = pair(x.x * c - x.y * s, x.x * s + x.y * c);
                        };
                        const float2 c0 = split(cs[0]), c1 = split(cs[1]), s0 = split(sn[0]), s1 = split(sn[1]);
                        turn(a0, c0.x, s0.x);
                        turn(a1, c0.y, s0.y);
                        turn(b0, c1.x, s1.x);
                        turn(b1, c1.y, s1.y);
                    } else {
                        const f32x2 u0 = fma2(b0, ms[0], mul2(a0, cs[0])), u1 = fma2(b1, ms[1], mul2(a1, cs[1]));
                        b0 = fma2(a0, sn[0], mul2(b0, cs[0]));
                        b1 = fma2(a1, sn[1], mul2(b1, cs[1]));
                        a0 = u0;
                        a1 = u1;
                    }
                }
                xa[i] = make_uint2(store2<T>(a0), store2<T>(a1));
                xb[i] = make_uint2(store2<T>(b0), store2<T>(b1));
            }
            if (row0 + i * RPW < rows) {
                *reinterpret_cast<uint2*>(dst + i * (RPW * dst_row) + da) = xa[i];
                *reinterpret_cast<uint2*>(dst + i * (RPW * dst_row) + db) = xb[i];
            }
        }
    }
}

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <typename T, int D, bool APPEND>
cudaError_t launch_rope(const RopeParams& p, bool inter, cudaStream_t st) {
    const dim3 grid(unsigned(((long long)p.stride * p.chunks + 3) / 4)), block(128);
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
    // One row group per warp while there are too few to fill the device, up to
    // kGroups beyond.
    const int rpw = 32 * 8 / D, gq = (a.hq + rpw - 1) / rpw, gk = (a.hkv + rpw - 1) / rpw;
    const long long per = (long long)a.tokens * (gq + (APPEND ? 2 : 1) * gk) / (152 * 32);
    p.per_chunk = int(per < 1 ? 1 : (per > kGroups ? kGroups : per));
    p.cq = (gq + p.per_chunk - 1) / p.per_chunk;
    p.ck = (gk + p.per_chunk - 1) / p.per_chunk;
    p.chunks = p.cq + (APPEND ? 2 : 1) * p.ck;
    // one wave of 8 CTAs of 4 warps per SM
    const int wave = 152 * 32 / p.chunks;
    p.stride = a.tokens < wave ? a.tokens : (wave < 1 ? 1 : wave);
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
