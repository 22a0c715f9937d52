// A KV cache in 4 bits: rows quantised as they are written, and blocks read
// back into a 16-bit cache.
//
// Mathematics. A row x is the D values of one token and kv head (K and V
// apart), of 16-bit type T:
//   lo = min x,  s = the smallest T not below fl32(fl32(max x - lo) / 15),
//   code = rne(fl32(x - lo) / s) in 0 .. 15 (0 where s = 0),
//   value = code s + lo, so |x - value| <= s / 2.
// lo is a value of the row, so T holds it exactly; s is rounded up, so that no
// code passes 15. A row of its own scale is final once written: other tokens of
// the block neither wait for it nor requantise it, one pass and one launch do.
// The quotient is decided exactly (the remainder of the nearest code, one fma,
// is compared with s / 2), so codes do not depend on how a division rounds.
//
// Layout: codes [blocks, kv heads, 16, D / 2] bytes, channel 2i in the low half
// of byte i; params [blocks, kv heads, 16] pairs (s, lo) of T. 4.25 bits a value
// at D = 128, 4.5 at D = 64.
//
// Both kernels move bytes: a group of D / 8 lanes takes a row of the write, 16
// bytes a lane; a lane of the read takes 4 bytes of codes and stores 16.
#include "common.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ write ---
struct U4Write {
    const uint16_t* src[2];      // K, V rows [tokens, hkv, D], `stride` values between tokens
    long long stride[2];
    uint32_t* codes[2];
    uint32_t* params[2];
    const int64_t* slots;
    uint32_t* status;
    long long pool_slots, rows;  // rows = tokens * 2 * hkv
    int hkv;
};

template <typename T>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    if constexpr (std::is_same<T, BF16>::value) {
        const __nv_bfloat162 r = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    } else {
        const __half2 r = __hmin2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
}
template <typename T>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    if constexpr (std::is_same<T, BF16>::value) {
        const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    } else {
        const __half2 r = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
}

// The smallest T not below x >= 0, as bits.
template <typename T>
__device__ __forceinline__ uint32_t round_up(float x) {
    if constexpr (std::is_same<T, BF16>::value) return __bfloat16_as_ushort(__float2bfloat16_ru(x));
    else return __half_as_ushort(__float2half_ru(x));
}

// rne(d / s) for 0 <= d, s > 0, the quotient exact: c is within one of it, and
// the remainder d - c s is exact in fp32 (d has 24 bits, s 11).
__device__ __forceinline__ uint32_t u4_code(float d, float s, float inv) {
    constexpr float kRound = 12582912.f;                 // 1.5 * 2^23: rounds to integers
    const float t = fmaf(d, inv, kRound);
    float c = t - kRound;
    const float r = fmaf(-c, s, d), r2 = 2.f * fabsf(r);
    if (r2 >= s) {                                       // at or beyond the border
        const bool odd = (__float_as_uint(t) & 1u) != 0;
        if (r2 > s || odd) c += r > 0.f ? 1.f : -1.f;
    }
    return __float_as_uint(c + kRound) & 15u;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) u4_write_kernel(const __grid_constant__ U4Write p) {
    constexpr int LPR = D / 8;                           // lanes per row
    griddep_wait();
    griddep_launch_dependents();
    const int col = threadIdx.x % LPR;
    const long long step = (long long)gridDim.x * (kThreads / LPR);
    for (long long r = (long long)blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR; r < p.rows; r += step) {
        const long long n = r / (2 * p.hkv);
        const int rem = int(r - n * (2 * p.hkv)), kv = rem >= p.hkv, h = kv ? rem - p.hkv : rem;
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(p.src[kv] + n * p.stride[kv] + (long long)h * D + 8 * col));
        const long long slot = __ldg(p.slots + n);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        uint32_t mn = min2<T>(min2<T>(w[0], w[1]), min2<T>(w[2], w[3]));
        uint32_t mx = max2<T>(max2<T>(w[0], w[1]), max2<T>(w[2], w[3]));
        // low half: the lane's minimum, high half: its maximum
        mn = min2<T>(mn, mn >> 16);
        mx = max2<T>(mx, mx << 16);
        const unsigned group = LPR == 32 ? kFull : ((1u << LPR) - 1) << ((threadIdx.x & 31) / LPR * LPR);
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) {
            mn = min2<T>(mn, __shfl_xor_sync(group, mn, o));
            mx = max2<T>(mx, __shfl_xor_sync(group, mx, o));
        }
        const float lo = unpack2(T{}, mn).x, hi = unpack2(T{}, mx).y;
        const uint32_t sbits = round_up<T>(__fdiv_rn(hi - lo, 15.f));
        const float s = unpack2(T{}, sbits).x;
        uint32_t word = 0;
        if (s > 0.f) {
            // below 2^-100 the reciprocal could overflow: such rows divide
            const bool tiny = s < 0x1p-100f;
            const float inv = tiny ? 0.f : __frcp_rn(s);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack2(T{}, w[i]);
                const float d0 = f.x - lo, d1 = f.y - lo;
                uint32_t c0, c1;
                if (!tiny) {
                    c0 = u4_code(d0, s, inv);
                    c1 = u4_code(d1, s, inv);
                } else {
                    c0 = uint32_t(__double2int_rn(double(d0) / double(s)));
                    c1 = uint32_t(__double2int_rn(double(d1) / double(s)));
                }
                word |= (c0 | c1 << 4) << (8 * i);
            }
        }
        if (slot < 0) continue;
        if (slot >= p.pool_slots) {
            if (col == 0) flag_status(p.status, PKV_DEV_BAD_SLOT);
            continue;
        }
        const long long row = ((slot / kBlockSize) * p.hkv + h) * kBlockSize + slot % kBlockSize;
        p.codes[kv][row * LPR + col] = word;
        if (col == 0) p.params[kv][row] = sbits | (mn << 16);
    }
}

// ------------------------------------------------------------------- read ---
struct U4Read {
    const uint32_t* codes[2];
    const uint32_t* params[2];
    uint4* out[2];
    const int32_t* src;
    const int32_t* dst;
    uint32_t* status;
    long long items;             // pairs * 2 * runs
    int runs;                    // runs of 128 words of codes per block
    int num_blocks, out_blocks;
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) u4_read_kernel(const __grid_constant__ U4Read p) {
    constexpr int LPR = D / 8;                           // words of codes per row
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long warps = (long long)gridDim.x * (kThreads / 32);
    for (long long item = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); item < p.items;
         item += warps) {
        const long long half = item / p.runs;
        const int run = int(item - half * p.runs), kv = int(half & 1);
        const int s = __ldg(p.src + (half >> 1)), d = __ldg(p.dst + (half >> 1));
        if (unsigned(s) >= unsigned(p.num_blocks) || unsigned(d) >= unsigned(p.out_blocks)) {
            if (lane == 0 && run == 0) flag_status(p.status, PKV_DEV_BAD_BLOCK);
            continue;
        }
        const long long from = ((long long)s * p.runs + run) * 128 + lane;
        const long long to = ((long long)d * p.runs + run) * 128 + lane;
        uint32_t w[4], q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = __ldg(p.codes[kv] + from + 32 * i);
            q[i] = __ldg(p.params[kv] + (from + 32 * i) / LPR);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 sl = unpack2(T{}, q[i]);
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float a = __uint_as_float(0x4b000000u | ((w[i] >> (8 * k)) & 15u)) - 8388608.f;
                const float b = __uint_as_float(0x4b000000u | ((w[i] >> (8 * k + 4)) & 15u)) - 8388608.f;
                o[k] = pack2<T>(fmaf(a, sl.x, sl.y), fmaf(b, sl.x, sl.y));
            }
            p.out[kv][to + 32 * i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Sizes and types that both calls check.
pkv_status check_cache(const pkv_cache_desc* c, pkv_dtype dtype) {
    if (!c || c->num_blocks <= 0 || c->num_kv_heads <= 0 || c->head_dim <= 0) return PKV_ERR_INVALID_ARG;
    if (c->kv_dtype != PKV_U4) return PKV_ERR_INVALID_ARG;
    if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
    if (c->block_size != kBlockSize || c->num_kv_heads > 0xffff) return PKV_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128) return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_u4_append(const void* k_new, int64_t k_stride, const void* v_new,
                                    int64_t v_stride, pkv_dtype src_dtype, int32_t num_tokens,
                                    const int64_t* slot_mapping, void* k_cache, void* v_cache,
                                    void* k_params, void* v_params, const pkv_cache_desc* cache,
                                    uint32_t* dev_status, cudaStream_t stream) {
    const pkv_status st = check_cache(cache, src_dtype);
    if (st != PKV_OK) return st;
    const int D = cache->head_dim, hkv = cache->num_kv_heads;
    if (num_tokens < 0 || k_stride < (long long)hkv * D || v_stride < (long long)hkv * D || k_stride % 8 ||
        v_stride % 8)
        return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    if (!k_new || !v_new || !slot_mapping || !k_cache || !v_cache || !k_params || !v_params)
        return PKV_ERR_INVALID_ARG;
    if (!aligned_to(k_new, 16) || !aligned_to(v_new, 16) || !aligned_to(slot_mapping, 8) ||
        !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || !aligned_to(k_params, 16) ||
        !aligned_to(v_params, 16) || !aligned_to(dev_status, 4))
        return PKV_ERR_INVALID_ARG;
    U4Write p;
    p.src[0] = static_cast<const uint16_t*>(k_new); p.src[1] = static_cast<const uint16_t*>(v_new);
    p.stride[0] = k_stride; p.stride[1] = v_stride;
    p.codes[0] = static_cast<uint32_t*>(k_cache); p.codes[1] = static_cast<uint32_t*>(v_cache);
    p.params[0] = static_cast<uint32_t*>(k_params); p.params[1] = static_cast<uint32_t*>(v_params);
    p.slots = slot_mapping; p.status = dev_status;
    p.pool_slots = (long long)cache->num_blocks * kBlockSize;
    p.rows = (long long)num_tokens * 2 * hkv;
    p.hkv = hkv;
    const long long per = kThreads / (D / 8), ctas = (p.rows + per - 1) / per;
    const dim3 grid(unsigned(ctas < 152 * 32 ? ctas : 152 * 32)), block(kThreads);
    cudaError_t e;
    if (src_dtype == PKV_BF16)
        e = D == 128 ? launch_pdl(u4_write_kernel<BF16, 128>, grid, block, 0, stream, p)
                     : launch_pdl(u4_write_kernel<BF16, 64>, grid, block, 0, stream, p);
    else
        e = D == 128 ? launch_pdl(u4_write_kernel<F16, 128>, grid, block, 0, stream, p)
                     : launch_pdl(u4_write_kernel<F16, 64>, grid, block, 0, stream, p);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

extern "C" pkv_status pkv_u4_read_blocks(const void* k_cache, const void* v_cache,
                                         const void* k_params, const void* v_params,
                                         const pkv_cache_desc* cache, const int32_t* src_blocks,
                                         pkv_dtype out_dtype, void* k_out, void* v_out,
                                         int32_t out_num_blocks, const int32_t* dst_blocks,
                                         int32_t num_pairs, uint32_t* dev_status,
                                         cudaStream_t stream) {
    const pkv_status st = check_cache(cache, out_dtype);
    if (st != PKV_OK) return st;
    if (num_pairs < 0 || out_num_blocks <= 0) return PKV_ERR_INVALID_ARG;
    if (num_pairs == 0) return PKV_OK;
    if (!k_cache || !v_cache || !k_params || !v_params || !src_blocks || !k_out || !v_out || !dst_blocks)
        return PKV_ERR_INVALID_ARG;
    if (!aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || !aligned_to(k_params, 16) ||
        !aligned_to(v_params, 16) || !aligned_to(k_out, 16) || !aligned_to(v_out, 16) ||
        !aligned_to(src_blocks, 4) || !aligned_to(dst_blocks, 4) || !aligned_to(dev_status, 4))
        return PKV_ERR_INVALID_ARG;
    const int D = cache->head_dim;
    U4Read p;
    p.codes[0] = static_cast<const uint32_t*>(k_cache); p.codes[1] = static_cast<const uint32_t*>(v_cache);
    p.params[0] = static_cast<const uint32_t*>(k_params); p.params[1] = static_cast<const uint32_t*>(v_params);
    p.out[0] = static_cast<uint4*>(k_out); p.out[1] = static_cast<uint4*>(v_out);
    p.src = src_blocks; p.dst = dst_blocks; p.status = dev_status;
    p.runs = cache->num_kv_heads * kBlockSize * (D / 8) / 128;
    p.items = (long long)num_pairs * 2 * p.runs;
    p.num_blocks = cache->num_blocks; p.out_blocks = out_num_blocks;
    const long long ctas = (p.items + kThreads / 32 - 1) / (kThreads / 32);
    const dim3 grid(unsigned(ctas < 152 * 32 ? ctas : 152 * 32)), block(kThreads);
    cudaError_t e;
    if (out_dtype == PKV_BF16)
        e = D == 128 ? launch_pdl(u4_read_kernel<BF16, 128>, grid, block, 0, stream, p)
                     : launch_pdl(u4_read_kernel<BF16, 64>, grid, block, 0, stream, p);
    else
        e = D == 128 ? launch_pdl(u4_read_kernel<F16, 128>, grid, block, 0, stream, p)
                     : launch_pdl(u4_read_kernel<F16, 64>, grid, block, 0, stream, p);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
