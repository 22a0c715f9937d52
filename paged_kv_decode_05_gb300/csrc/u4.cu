// A KV cache in 4 bits: rows quantised as they are written, and blocks read
// back into a 16-bit cache.
//
// Mathematics. A row x is the D values of one token and kv head (K and V
// apart), of 16-bit type T:
//   lo = min x,  s = the smallest T not below fl32(fl32(max x - lo) / 15),
//   or the T below that where fl32(15 s + lo) passes T's largest value,
//   code = rne(fl32(x - lo) / s) in 0 .. 15 (0 where s = 0),
//   value = code s + lo, so |x - value| <= s / 2.
// lo is a value of the row, so T holds it exactly; s is rounded up, so that no
// quotient passes 15. Beside T's largest value the top code could then stand for
// more than T holds (fp16, 0 to 65504: s = 4368, 15 s = 65520, infinity when read
// back); rounded down there, the quotient of the row's maximum is at most
// 15 (1 + 2^-7), still code 15. A row of its own scale is final once written: other
// tokens of the block neither wait for it nor requantise it, one pass and one launch do.
// The quotient is decided exactly (the remainder of the nearest code, one fma,
// is compared with s / 2), so codes do not depend on how a division rounds.
//
// Layout: codes [blocks, kv heads, 16, D / 2] bytes, channel 2i in the low half
// of byte i; params [blocks, kv heads, 16] pairs (s, lo) of T. 4.25 bits a value
// at D = 128, 4.5 at D = 64.
//
// Both kernels move bytes: D / 16 lanes take a row of the write, twice 16 bytes a lane;
// a lane of the read takes 4 bytes of codes and stores 16 (streaming: the cache it fills is
// larger than what L2 would keep for the reader).
//
// Measured (8 kv heads, D = 128, bf16): 8192 tokens written in 17 us with cold caches
// (50 MB, 2.5 TB/s: the issue slots are 0.72 busy, minimum, maximum and an exact quotient
// for every value; 8 values a lane 25.6), 256 tokens in 5.6; 8192 blocks read back in
// 112 us (0.68 GB at 0.89 of the copy rate: memory; without streaming stores 117).
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
    long long pool_slots;
    int tokens, hkv;
    int groups;                  // warps that share a token's 2 hkv rows
    int every;                   // tokens between a warp's
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

// A row's scale, as bits.
template <typename T>
__device__ __forceinline__ uint32_t u4_scale(float lo, float hi) {
    constexpr float kMost = std::is_same<T, BF16>::value ? 0x1.fep127f : 65504.f;
    const uint32_t s = round_up<T>(__fdiv_rn(hi - lo, 15.f));
    return s - (hi <= kMost && fmaf(15.f, unpack2(T{}, s).x, lo) > kMost ? 1u : 0u);
}

// Codes rne((x - lo) / s) of 8 values, packed; inv is 1 / s but for the last bits, or 0
// where it could overflow. A product with inv lands within one of each code; the
// remainders r = d - c s are exact in fp32 (d has 24 bits, s 11), and a code whose
// remainder passes s / 2, or meets it while odd, gives way to its neighbour. (Such ties
// are common between numbers of 8 bits: one value in 420, one row in 4.)
template <typename T>
__device__ __forceinline__ uint32_t u4_codes(const uint4& x, float lo, float s, float inv) {
    constexpr float kRound = 12582912.f;                 // 1.5 * 2^23: rounds to integers
    constexpr uint32_t kBits = 0x4b400000u * 0x11111111u;    // its bits at the 8 places, which go again
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t word = 0u - kBits;
    if (inv != 0.f) {
        float r[8], worst = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = unpack2(T{}, w[i / 2]);
            const float d = (i & 1 ? f.y : f.x) - lo;
            const float t = fmaf(d, inv, kRound);
            r[i] = fmaf(kRound - t, s, d);
            worst = fmaxf(worst, fabsf(r[i]));
            word += __float_as_uint(t) << (4 * i);
        }
        if (2.f * worst >= s) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float r2 = 2.f * fabsf(r[i]);
                if (r2 > s || (r2 == s && (word >> (4 * i) & 1u)))
                    word += r[i] > 0.f ? 1u << (4 * i) : 0u - (1u << (4 * i));
            }
        }
        return word;
    }
    word = 0u;
    for (int i = 0; s > 0.f && i < 8; ++i) {
        const float2 f = unpack2(T{}, w[i / 2]);
        const float d = (i & 1 ? f.y : f.x) - lo;
        word |= (uint32_t(__double2int_rn(double(d) / double(s))) & 15u) << (4 * i);
    }
    return word;
}

// A warp takes one group of 4 (D = 128) or 8 (D = 64) of a token's 2 hkv rows, K's and
// then V's, and every `every`-th token, whose rows it reads one token ahead. A lane has
// two runs of 8 values, half a row apart, which share the row's maximum, minimum and
// divisions.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) u4_write_kernel(const __grid_constant__ U4Write p) {
    constexpr int LPR = D / 16, RPW = 32 / LPR;          // lanes per row, rows per warp
    constexpr int WPR = D / 8;                           // words of codes per row
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, col = lane % LPR;
    const int wid = int(blockIdx.x) * (kThreads / 32) + int(threadIdx.x >> 5);
    const int n0 = wid / p.groups, row = (wid - n0 * p.groups) * RPW + lane / LPR;
    if (n0 >= p.every || n0 >= p.tokens) return;        // the whole warp
    const bool have = row < 2 * p.hkv;                   // a group may end past the rows
    const int kv = have && row >= p.hkv, h = have ? row - kv * p.hkv : 0;
    const uint16_t* src = p.src[kv] + h * D + 8 * col;
    uint32_t* codes = p.codes[kv] + (long long)h * (kBlockSize * WPR) + col;
    uint32_t* params = p.params[kv] + (long long)h * kBlockSize;
    const long long step = p.stride[kv];
    uint4 x0 = __ldg(reinterpret_cast<const uint4*>(src + n0 * step));
    uint4 x1 = __ldg(reinterpret_cast<const uint4*>(src + n0 * step + D / 2));
    long long slot = __ldg(p.slots + n0);
    for (int n = n0;;) {
        const uint4 a = x0, b = x1;
        const long long at = slot;
        const long long next = (long long)n + p.every;
        if (next < p.tokens) {
            x0 = __ldg(reinterpret_cast<const uint4*>(src + next * step));
            x1 = __ldg(reinterpret_cast<const uint4*>(src + next * step + D / 2));
            slot = __ldg(p.slots + next);
        }
        uint32_t mn = min2<T>(min2<T>(min2<T>(a.x, a.y), min2<T>(a.z, a.w)),
                              min2<T>(min2<T>(b.x, b.y), min2<T>(b.z, b.w)));
        uint32_t mx = max2<T>(max2<T>(max2<T>(a.x, a.y), max2<T>(a.z, a.w)),
                              max2<T>(max2<T>(b.x, b.y), max2<T>(b.z, b.w)));
        // low half: the lane's minimum, high half: its maximum
        mn = min2<T>(mn, mn >> 16);
        mx = max2<T>(mx, mx << 16);
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) {
            mn = min2<T>(mn, __shfl_xor_sync(kFull, mn, o));
            mx = max2<T>(mx, __shfl_xor_sync(kFull, mx, o));
        }
        const float lo = unpack2(T{}, mn).x, hi = unpack2(T{}, mx).y;
        const uint32_t sbits = u4_scale<T>(lo, hi);
        const float s = unpack2(T{}, sbits).x;
        float inv = 0.f;
        if (s >= 0x1p-100f) asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(s));
        const uint32_t c0 = u4_codes<T>(a, lo, s, inv), c1 = u4_codes<T>(b, lo, s, inv);
        if (have && at >= 0) {
            if (at < p.pool_slots) {
                const uint32_t blk = uint32_t(at >> 4), r = uint32_t(at) & (kBlockSize - 1);
                const long long tile = (long long)blk * p.hkv;
                uint32_t* to = codes + (tile * kBlockSize + r) * WPR;
                to[0] = c0;
                to[WPR / 2] = c1;
                if (col == 0) params[tile * kBlockSize + r] = sbits | (mn << 16);
            } else if (col == 0) {
                flag_status(p.status, PKV_DEV_BAD_SLOT);
            }
        }
        if (next >= p.tokens) break;
        n = int(next);
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
    int pairs, runs;             // runs of 128 words of codes per block
    int num_blocks, out_blocks;
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) u4_read_kernel(const __grid_constant__ U4Read p) {
    constexpr int LPR = D / 8;                           // words of codes per row
    griddep_wait();
    griddep_launch_dependents();
    // a warp takes one run of K or V, and every step-th pair
    const int lane = threadIdx.x & 31;
    const long long warps = (long long)gridDim.x * (kThreads / 32);
    const long long wid = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int per = 2 * p.runs, step = int(warps / per);
    if (wid >= (long long)step * per) return;
    const int pair0 = int(wid / per), part = int(wid - (long long)pair0 * per);
    const int kv = part >= p.runs, run = part - kv * p.runs;
    for (long long pair = pair0; pair < p.pairs; pair += step) {
        const int s = __ldg(p.src + pair), d = __ldg(p.dst + pair);
        if (unsigned(s) >= unsigned(p.num_blocks) || unsigned(d) >= unsigned(p.out_blocks)) {
            if (lane == 0 && part == 0) flag_status(p.status, PKV_DEV_BAD_BLOCK);
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
            __stcs(p.out[kv] + to + 32 * i, make_uint4(o[0], o[1], o[2], o[3]));
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
    p.tokens = num_tokens;
    p.hkv = hkv;
    const int rpw = 512 / D;
    p.groups = (2 * hkv + rpw - 1) / rpw;
    // two waves of 8 CTAs per SM at most
    const int most = 152 * 2 * kThreads / 32 * 8 / p.groups;
    p.every = num_tokens < most ? num_tokens : (most < 1 ? 1 : most);
    const long long warps = (long long)p.every * p.groups;
    const dim3 grid(unsigned((warps + kThreads / 32 - 1) / (kThreads / 32))), block(kThreads);
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
    p.pairs = num_pairs;
    p.num_blocks = cache->num_blocks; p.out_blocks = out_num_blocks;
    // at least one warp for each run, at most 32 CTAs per SM in turn
    const long long per = 2ll * p.runs, most = 152ll * 32 * kThreads / 32 / per;
    const long long warps = per * (num_pairs < most ? num_pairs : (most < 1 ? 1 : most));
    const dim3 grid(unsigned((warps + kThreads / 32 - 1) / (kThreads / 32))), block(kThreads);
    cudaError_t e;
    if (out_dtype == PKV_BF16)
        e = D == 128 ? launch_pdl(u4_read_kernel<BF16, 128>, grid, block, 0, stream, p)
                     : launch_pdl(u4_read_kernel<BF16, 64>, grid, block, 0, stream, p);
    else
        e = D == 128 ? launch_pdl(u4_read_kernel<F16, 128>, grid, block, 0, stream, p)
                     : launch_pdl(u4_read_kernel<F16, 64>, grid, block, 0, stream, p);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
