// The cheap choice of blocks for sparse decode attention: channel bounds of a
// block's keys, an upper bound of every block's scores, and the best blocks.
#include "choose.cuh"

namespace pkv {
namespace {

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

pkv_status check_desc(const pkv_cache_desc* c) {
    if (!c || c->num_blocks <= 0 || c->num_kv_heads <= 0 || c->head_dim <= 0) return PKV_ERR_INVALID_ARG;
    if (c->kv_dtype != PKV_F16 && c->kv_dtype != PKV_BF16 && c->kv_dtype != PKV_I8)
        return PKV_ERR_INVALID_ARG;
    if (c->block_size != kBlockSize || (c->head_dim != 64 && c->head_dim != 128))
        return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

// ---------------------------------------------------------------- bounds ---
// lo_d = min_t k_td, hi_d = max_t k_td over the valid rows of a block: one
// warp per (sequence, block, kv head), one 16-byte load per lane and row.
// Bound by memory: a tile is read and two rows are written.
struct BoundsParams {
    const unsigned char* k_cache;
    unsigned char* bounds;        // [num_blocks, hkv, 2, D]: min, max
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* num_new;       // [batch] or nullptr (1 each)
    uint32_t* status;
    int batch, hkv, mb, num_blocks, max_new, span;
};

template <typename KV>
__device__ __forceinline__ uint32_t min_word(uint32_t a, uint32_t b) {
    if constexpr (std::is_same<KV, I8>::value) return __vmins4(a, b);
    else if constexpr (std::is_same<KV, BF16>::value) {
        const __nv_bfloat162 r = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    } else {
        const __half2 r = __hmin2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
}
template <typename KV>
__device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b) {
    if constexpr (std::is_same<KV, I8>::value) return __vmaxs4(a, b);
    else if constexpr (std::is_same<KV, BF16>::value) {
        const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    } else {
        const __half2 r = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
}

template <typename KV, int D>
__global__ void __launch_bounds__(256) block_bounds_kernel(const BoundsParams p) {
    constexpr int ROW = D * Elem<KV>::bytes;
    constexpr int LPR = ROW / 16;            // lanes per row
    constexpr int RG = 32 / LPR;             // rows read side by side
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, col = lane % LPR, rg = lane / LPR;
    const long long items = (long long)p.batch * p.span * p.hkv;
    for (long long it = (blockIdx.x * (long long)blockDim.x + threadIdx.x) >> 5; it < items;
         it += ((long long)gridDim.x * blockDim.x) >> 5) {
        const int kvh = int(it % p.hkv);
        const long long r = it / p.hkv;
        const int jj = int(r % p.span), b = int(r / p.span);
        const int L = p.context_lens[b];
        const int n = p.num_new ? p.num_new[b] : (L > 0 ? 1 : 0);
        if (L < 0 || L > (long long)p.mb * kBlockSize || n < 0 || n > p.max_new || n > L) {
            if (jj == 0 && kvh == 0 && lane == 0) flag_status(p.status, PKV_DEV_BAD_LENGTH);
            continue;
        }
        const int j = (L - n) / kBlockSize + jj;
        if (n == 0 || j * kBlockSize >= L) continue;
        const int blk = p.block_tables[(long long)b * p.mb + j];
        if (unsigned(blk) >= unsigned(p.num_blocks)) {
            if (kvh == 0 && lane == 0) flag_status(p.status, PKV_DEV_BAD_BLOCK);
            continue;
        }
        const int nv = min(kBlockSize, L - j * kBlockSize);
        const long long tile = (long long)blk * p.hkv + kvh;
        const unsigned char* src = p.k_cache + tile * kBlockSize * ROW + col * 16;
        uint4 x[kBlockSize / RG];
#pragma unroll
        for (int i = 0; i < kBlockSize / RG; ++i) {
            // rows past the valid ones repeat row 0, which changes neither bound
            const int row = rg + i * RG;
            x[i] = *reinterpret_cast<const uint4*>(src + (row < nv ? row : 0) * ROW);
        }
        uint32_t lo[4] = {x[0].x, x[0].y, x[0].z, x[0].w}, hi[4] = {x[0].x, x[0].y, x[0].z, x[0].w};
#pragma unroll
        for (int i = 1; i < kBlockSize / RG; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                lo[c] = min_word<KV>(lo[c], w[c]);
                hi[c] = max_word<KV>(hi[c], w[c]);
            }
        }
#pragma unroll
        for (int off = LPR; off < 32; off <<= 1)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                lo[c] = min_word<KV>(lo[c], __shfl_xor_sync(kFull, lo[c], off));
                hi[c] = max_word<KV>(hi[c], __shfl_xor_sync(kFull, hi[c], off));
            }
        unsigned char* dst = p.bounds + tile * 2 * ROW + col * 16;
        if (rg == 0) *reinterpret_cast<uint4*>(dst) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        if (rg == RG - 1) *reinterpret_cast<uint4*>(dst + ROW) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    }
}

// ---------------------------------------------------------------- scores ---
// score = max over the group's heads of sum_d max(q_d lo_d, q_d hi_d). Since
// max(q lo, q hi) = min(q, 0) lo + max(q, 0) hi, it is a product over 2 D
// terms of the block's bounds with (min(q, 0), max(q, 0)): 16 blocks are the
// rows and the heads the columns of mma.sync m16n8k16, fed from global memory
// (each bound is used once, so shared memory would add nothing). Four
// accumulators share the 2 D terms and are added in fp32. Bound by memory:
// 2 D elements per (block, kv head), 1/16 of what attention over it reads.
// One factor of each pair is zero, so an infinite bound (a key that overflowed)
// makes a sum NaN that need not be: a run with such a sum is scored again, term
// by term (exact_score; after the loop, inside it the call cost 4 %). INT8 codes
// meet q in fp16: a bf16 head is brought into its range by a power of two.
struct ScoreParams {
    const void* q;
    const unsigned char* bounds;
    const float* k_scales;
    const int32_t* block_tables;
    const int32_t* context_lens;
    float* scores;               // [batch, hkv, mb]
    uint32_t* status;
    int batch, hq, hkv, mb, num_blocks;
    int groups;                  // runs of kScoreRun blocks of a row, one warp each
};

// Warps per CTA, and blocks per warp (2 tiles of 16 under one set of query
// fragments): short warps in small CTAs spread best over the SMs. 32 sequences
// of 8k to 32k tokens and 3 of up to 3000, the bounds of the newest blocks
// included: 31.5 and 5.2 us, against 33.7 and 7.1 with 64 blocks and 8 warps; a
// ring of cp.async tiles per warp was slower (41 us): many warps hide the
// latency better than a long queue in a few.
constexpr int kScoreWarps = 4;
constexpr int kScoreRun = 32;

// Negative (sign = true) or positive parts of two packed 16-bit values; NaN stays in one.
template <typename QT>
__device__ __forceinline__ uint32_t part2(uint32_t w, bool neg) {
    const float2 f = unpack2(QT{}, w);
    return neg ? pack2<QT>(fminf(f.x, 0.f), fminf(f.y, 0.f))
               : pack2<QT>(f.x < 0.f ? 0.f : f.x, f.y < 0.f ? 0.f : f.y);
}

// a b, where nothing times infinity is nothing.
__device__ __forceinline__ float times(float a, float b) {
    const float x = a * b;
    return x != x && a == a && b == b ? 0.f : x;
}

__device__ __forceinline__ float load_code(const unsigned char* p) { return float(int8_t(*p)); }

// The score of one block (bounds at `box`) for G heads of q, term by term by one
// warp; a head whose sum is not a number does not count.
template <typename KV, typename QT, int D, int G>
__device__ __noinline__ float exact_score(const uint16_t* q, const unsigned char* box) {
    const int lane = threadIdx.x & 31;
    float best = -INFINITY;
    for (int h = 0; h < G; ++h) {
        float s = 0.f;
        for (int d = lane; d < D; d += 32) {
            const float x = load_scalar(QT{}, q, h * D + d);
            float lo, hi;
            if constexpr (std::is_same<KV, I8>::value) {
                lo = load_code(box + d);
                hi = load_code(box + D + d);
            } else {
                lo = load_scalar(KV{}, box, d);
                hi = load_scalar(KV{}, box, D + d);
            }
            s += fmaxf(times(x, lo), times(x, hi));
        }
#pragma unroll
        for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(kFull, s, off);
        best = fmaxf(best, s);
    }
    return best;
}

__device__ __forceinline__ uint32_t codes2(uint32_t biased, uint32_t sel) {   // exact fp16 codes
    const uint32_t w = i8x2_biased_h2(biased, sel);
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&w), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t*>(&r);
}

template <typename KV, typename QT, int D, int G>
__global__ void __launch_bounds__(32 * kScoreWarps, 4) block_scores_kernel(const ScoreParams p) {
    constexpr bool I = std::is_same<KV, I8>::value;
    using MT = typename std::conditional<I, F16, KV>::type;
    constexpr int ROW = 2 * D * Elem<KV>::bytes;     // lo and hi of one block
    constexpr int NK = 2 * D / 16;                   // k-steps; the first half meets lo
    constexpr int NC = ROW / 64;                     // 64-byte spans, 16 bytes a lane
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gq = lane >> 2, tq = lane & 3;
    const long long items = (long long)p.batch * p.hkv * p.groups;
    const long long it = (long long)blockIdx.x * kScoreWarps + warp;
    if (it >= items) return;
    const long long seg = it / p.groups;
    const int j0 = int(it - seg * p.groups) * kScoreRun;
    const int b = int(seg / p.hkv), kvh = int(seg - (long long)b * p.hkv);
    int L = p.context_lens[b];
    if (L < 0 || L > (long long)p.mb * kBlockSize) {
        if (j0 == 0 && kvh == 0 && lane == 0) flag_status(p.status, PKV_DEV_BAD_LENGTH);
        L = L < 0 ? 0 : p.mb * kBlockSize;
    }
    const int nblk = (L + kBlockSize - 1) / kBlockSize, j1 = min(j0 + kScoreRun, p.mb);
    float* out = p.scores + seg * p.mb;
    for (int j = max(j0, nblk) + lane; j < j1; j += 32) out[j] = -INFINITY;
    if (j0 >= nblk) return;
    // the run's physical blocks, one per lane (-1: none, flagged)
    int tab[kScoreRun / 32];
#pragma unroll
    for (int i = 0; i < kScoreRun / 32; ++i) {
        const int j = j0 + 32 * i + lane;
        tab[i] = j < nblk ? __ldg(p.block_tables + (long long)b * p.mb + j) : -1;
        if (j < nblk && unsigned(tab[i]) >= unsigned(p.num_blocks)) {
            if (kvh == 0) flag_status(p.status, PKV_DEV_BAD_BLOCK);
            tab[i] = -1;
        }
    }
    // B fragments, the contraction index permuted so that a lane's 16 bytes
    // serve whole k-steps: 16-bit k-steps 2c, 2c + 1 take dims 32c + 8tq +
    // [0, 4) and + [4, 8); INT8 k-steps 4c + k take dims 64c + 16tq + 4k + [0, 4).
    const uint16_t* qrow = static_cast<const uint16_t*>(p.q) + ((long long)b * p.hq + kvh * G + gq) * D;
    uint32_t qb[NK][2];
    constexpr bool FIT = I && std::is_same<QT, BF16>::value;
    float up[2] = {1.f, 1.f};          // FIT: what heads 2tq, 2tq + 1 were divided by
    uint2 w[NK / 2];
    float amax = 0.f;
#pragma unroll
    for (int ks = 0; ks < NK / 2; ++ks) {
        const int d0 = I ? 64 * (ks / 4) + 16 * tq + 4 * (ks % 4) : 32 * (ks / 2) + 8 * tq + 4 * (ks % 2);
        w[ks] = make_uint2(0u, 0u);
        if (gq < G) w[ks] = __ldg(reinterpret_cast<const uint2*>(qrow + d0));
        if constexpr (FIT) {
            const float2 f0 = unpack2(QT{}, w[ks].x), f1 = unpack2(QT{}, w[ks].y);
            amax = fmaxf(fmaxf(fmaxf(amax, fabsf(f0.x)), fmaxf(fabsf(f0.y), fabsf(f1.x))), fabsf(f1.y));
        }
    }
    if constexpr (FIT) {               // a head's dims lie in lanes 4 gq + [0, 4)
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
        const float2 fit = fit_half(amax);
#pragma unroll
        for (int ks = 0; ks < NK / 2; ++ks) {
            const float2 f0 = unpack2(QT{}, w[ks].x), f1 = unpack2(QT{}, w[ks].y);
            w[ks] = make_uint2(pack2<F16>(f0.x * fit.x, f0.y * fit.x), pack2<F16>(f1.x * fit.x, f1.y * fit.x));
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) up[e] = __shfl_sync(kFull, fit.y, (8 * tq + 4 * e) & 31);
    }
#pragma unroll
    for (int ks = 0; ks < NK / 2; ++ks) {
        qb[ks][0] = part2<MT>(w[ks].x, true);
        qb[ks][1] = part2<MT>(w[ks].y, true);
        qb[NK / 2 + ks][0] = part2<MT>(w[ks].x, false);
        qb[NK / 2 + ks][1] = part2<MT>(w[ks].y, false);
    }
    bool odd = false;                  // some sum is NaN
#pragma unroll 1
    for (int jt = j0; jt < min(j1, nblk); jt += 16) {
        // rows gq and gq + 8 of the tile: blocks jt + gq, jt + gq + 8
        int blk[2];
        uint4 x[2][NC];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int k = jt - j0 + gq + 8 * r;
            int v = __shfl_sync(kFull, tab[0], k & 31);
#pragma unroll
            for (int i = 1; i < kScoreRun / 32; ++i) {
                const int y = __shfl_sync(kFull, tab[i], k & 31);
                if (k >= 32 * i) v = y;
            }
            blk[r] = v;
            const unsigned char* src = p.bounds + ((long long)max(v, 0) * p.hkv + kvh) * ROW + 16 * tq;
#pragma unroll
            for (int c = 0; c < NC; ++c) x[r][c] = __ldcs(reinterpret_cast<const uint4*>(src + 64 * c));
        }
        float acc[4][4];
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[c][0] = acc[c][1] = acc[c][2] = acc[c][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < NK; ++kk) {
            uint32_t a[4];
            if constexpr (!I) {
                const uint4 x0 = x[0][kk / 2], x1 = x[1][kk / 2];
                if (kk % 2 == 0) { a[0] = x0.x; a[1] = x1.x; a[2] = x0.y; a[3] = x1.y; }
                else { a[0] = x0.z; a[1] = x1.z; a[2] = x0.w; a[3] = x1.w; }
            } else {
                const uint4 x0 = x[0][kk / 4], x1 = x[1][kk / 4];
                const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w1[4] = {x1.x, x1.y, x1.z, x1.w};
                const uint32_t y0 = w0[kk % 4] ^ 0x80808080u, y1 = w1[kk % 4] ^ 0x80808080u;
                a[0] = codes2(y0, 0x4140); a[1] = codes2(y1, 0x4140);
                a[2] = codes2(y0, 0x4342); a[3] = codes2(y1, 0x4342);
            }
            mma16816<MT>(acc[kk % 4], a, qb[kk][0], qb[kk][1]);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float best = -INFINITY, all = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float s = (acc[0][2 * r + e] + acc[1][2 * r + e]) + (acc[2][2 * r + e] + acc[3][2 * r + e]);
                if constexpr (FIT) s *= up[e];
                if (2 * tq + e < G) {
                    best = fmaxf(best, s);
                    all += s;
                }
            }
            best = fmaxf(best, __shfl_xor_sync(kFull, best, 1));
            best = fmaxf(best, __shfl_xor_sync(kFull, best, 2));
            odd = odd || (all != all && blk[r] >= 0);
            const int j = jt + gq + 8 * r;
            if (tq == 0 && j < nblk) {
                float s = -INFINITY;
                if (blk[r] >= 0) {
                    s = best;
                    if constexpr (I) s *= __ldg(p.k_scales + (long long)blk[r] * p.hkv + kvh);
                }
                out[j] = s;
            }
        }
    }
    if (!__any_sync(kFull, odd)) return;
    __syncwarp();                      // the scores below replace other lanes' ones
    for (int k = 0; k < kScoreRun; ++k) {
        static_assert(kScoreRun == 32, "a block per lane");
        const int v = __shfl_sync(kFull, tab[0], k);
        if (v < 0) continue;
        float s = exact_score<KV, QT, D, G>(
            static_cast<const uint16_t*>(p.q) + ((long long)b * p.hq + kvh * G) * D,
            p.bounds + ((long long)v * p.hkv + kvh) * ROW);
        if constexpr (I) s *= __ldg(p.k_scales + (long long)v * p.hkv + kvh);
        if (lane == 0) out[j0 + k] = s;
    }
}

// ---------------------------------------------------------------- select ---
// One CTA per (sequence, kv head) (see choose.cuh). Rows of up to choose::kKeepRow
// scores are kept in shared memory between the passes.
struct SelectParams {
    const float* scores;         // [batch, hkv, mb]
    const int32_t* context_lens;
    int32_t* lists;              // [batch, hkv, budget]
    int32_t* list_lens;          // [batch]
    uint32_t* status;
    int hkv, mb, budget, keep_first, keep_last, cap;   // cap: scores the shared row holds
};

template <int T>
__global__ void __launch_bounds__(T, 1536 / T) block_select_kernel(const SelectParams p) {
    extern __shared__ uint32_t row[];
    __shared__ choose::Scratch<T> s;
    griddep_wait();
    griddep_launch_dependents();
    const int seg = blockIdx.x, b = seg / p.hkv, kvh = seg - b * p.hkv;
    int L = p.context_lens[b];
    if (L < 0 || L > (long long)p.mb * kBlockSize) {
        if (kvh == 0 && threadIdx.x == 0) flag_status(p.status, PKV_DEV_BAD_LENGTH);
        L = L < 0 ? 0 : p.mb * kBlockSize;
    }
    const int n = (L + kBlockSize - 1) / kBlockSize, count = min(n, p.budget);
    const float* src = p.scores + (long long)seg * p.mb;
    int32_t* out = p.lists + (long long)seg * p.budget;
    if (kvh == 0 && threadIdx.x == 0) p.list_lens[b] = count;
    for (int i = count + threadIdx.x; i < p.budget; i += T) out[i] = -1;
    if (count == n) {
        for (int i = threadIdx.x; i < n; i += T) out[i] = i;
        return;
    }
    choose::choose_row<T>(s, [&](int i) { return __ldcg(src + i); }, n <= p.cap ? row : nullptr, n,
                          p.keep_first, p.keep_last, count,
                          [&](int rank, int i, uint32_t) { out[rank] = i; });
}

template <int T>
cudaError_t launch_select(const SelectParams& p, int rows, cudaStream_t st) {
    return choose::launch_rows<block_select_kernel<T>, T>(p, rows, st);
}

template <typename KV, typename QT, int D>
cudaError_t launch_scores(const ScoreParams& p, int G, cudaStream_t st) {
    const long long items = (long long)p.batch * p.hkv * p.groups;
    const dim3 grid(unsigned((items + kScoreWarps - 1) / kScoreWarps)), block(32 * kScoreWarps);
    switch (G) {
        case 1: return launch_pdl(block_scores_kernel<KV, QT, D, 1>, grid, block, 0, st, p);
        case 2: return launch_pdl(block_scores_kernel<KV, QT, D, 2>, grid, block, 0, st, p);
        case 4: return launch_pdl(block_scores_kernel<KV, QT, D, 4>, grid, block, 0, st, p);
        default: return launch_pdl(block_scores_kernel<KV, QT, D, 8>, grid, block, 0, st, p);
    }
}

template <typename KV, typename QT>
cudaError_t launch_scores(const ScoreParams& p, int D, int G, cudaStream_t st) {
    return D == 128 ? launch_scores<KV, QT, 128>(p, G, st) : launch_scores<KV, QT, 64>(p, G, st);
}

template <typename KV>
cudaError_t launch_bounds(const BoundsParams& p, int D, cudaStream_t st) {
    const long long items = (long long)p.batch * p.span * p.hkv;
    long long grid = (items + 7) / 8;
    if (grid > (1 << 20)) grid = 1 << 20;
    return D == 128 ? launch_pdl(block_bounds_kernel<KV, 128>, dim3(unsigned(grid)), dim3(256), 0, st, p)
                    : launch_pdl(block_bounds_kernel<KV, 64>, dim3(unsigned(grid)), dim3(256), 0, st, p);
}

pkv_status done(cudaError_t e) {
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_block_bounds(const void* k_cache, const pkv_cache_desc* cache,
                                       const int32_t* block_tables, int32_t max_blocks_per_seq,
                                       const int32_t* context_lens, const int32_t* num_new,
                                       int32_t max_new, int32_t batch, void* bounds,
                                       uint32_t* dev_status, cudaStream_t stream) {
    const pkv_status s = check_desc(cache);
    if (s != PKV_OK) return s;
    if (batch < 0 || max_new < 0 || max_blocks_per_seq <= 0 ||
        max_blocks_per_seq > 0x7fffffff / kBlockSize || (!num_new && max_new != 1))
        return PKV_ERR_INVALID_ARG;
    if (batch == 0 || max_new == 0) return PKV_OK;
    if (!k_cache || !block_tables || !context_lens || !bounds) return PKV_ERR_INVALID_ARG;
    if (!aligned_to(k_cache, 16) || !aligned_to(bounds, 16) || !aligned_to(block_tables, 4) ||
        !aligned_to(context_lens, 4) || !aligned_to(num_new, 4) || !aligned_to(dev_status, 4))
        return PKV_ERR_INVALID_ARG;
    BoundsParams p;
    p.k_cache = static_cast<const unsigned char*>(k_cache);
    p.bounds = static_cast<unsigned char*>(bounds);
    p.block_tables = block_tables; p.context_lens = context_lens; p.num_new = num_new;
    p.status = dev_status;
    p.batch = batch; p.hkv = cache->num_kv_heads; p.mb = max_blocks_per_seq;
    p.num_blocks = cache->num_blocks; p.max_new = max_new;
    // blocks that max_new consecutive positions can touch
    const long long span = ((long long)max_new + kBlockSize - 2) / kBlockSize + 1;
    p.span = int(span < p.mb ? span : p.mb);
    const int D = cache->head_dim;
    return done(cache->kv_dtype == PKV_BF16  ? launch_bounds<BF16>(p, D, stream)
                : cache->kv_dtype == PKV_F16 ? launch_bounds<F16>(p, D, stream)
                                             : launch_bounds<I8>(p, D, stream));
}

extern "C" pkv_status pkv_block_scores(const void* q, pkv_dtype q_dtype, const void* bounds,
                                       const float* k_scales, const pkv_cache_desc* cache,
                                       const int32_t* block_tables, int32_t max_blocks_per_seq,
                                       const int32_t* context_lens, int32_t batch,
                                       int32_t num_q_heads, float* scores, uint32_t* dev_status,
                                       cudaStream_t stream) {
    const pkv_status s = check_desc(cache);
    if (s != PKV_OK) return s;
    if (q_dtype != PKV_F16 && q_dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
    if (cache->kv_dtype != PKV_I8 && q_dtype != cache->kv_dtype) return PKV_ERR_INVALID_ARG;
    if (batch < 0 || max_blocks_per_seq <= 0 || max_blocks_per_seq > 0x7fffffff / kBlockSize ||
        num_q_heads <= 0 || num_q_heads % cache->num_kv_heads)
        return PKV_ERR_INVALID_ARG;
    const int G = num_q_heads / cache->num_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8) return PKV_ERR_UNSUPPORTED;
    if (batch == 0) return PKV_OK;
    if (!q || !bounds || !block_tables || !context_lens || !scores) return PKV_ERR_INVALID_ARG;
    if (!aligned_to(q, 16) || !aligned_to(bounds, 16) || !aligned_to(block_tables, 4) ||
        !aligned_to(context_lens, 4) || !aligned_to(scores, 4) || !aligned_to(dev_status, 4))
        return PKV_ERR_INVALID_ARG;
    if (cache->kv_dtype == PKV_I8 && (!k_scales || !aligned_to(k_scales, 4))) return PKV_ERR_INVALID_ARG;
    ScoreParams p;
    p.q = q; p.bounds = static_cast<const unsigned char*>(bounds); p.k_scales = k_scales;
    p.block_tables = block_tables; p.context_lens = context_lens; p.scores = scores;
    p.status = dev_status;
    p.batch = batch; p.hq = num_q_heads; p.hkv = cache->num_kv_heads; p.mb = max_blocks_per_seq;
    p.num_blocks = cache->num_blocks;
    p.groups = (max_blocks_per_seq + kScoreRun - 1) / kScoreRun;
    if (((long long)batch * p.hkv * p.groups + kScoreWarps - 1) / kScoreWarps > 0x7fffffffLL)
        return PKV_ERR_UNSUPPORTED;
    const int D = cache->head_dim;
    cudaError_t e;
    if (cache->kv_dtype == PKV_BF16) e = launch_scores<BF16, BF16>(p, D, G, stream);
    else if (cache->kv_dtype == PKV_F16) e = launch_scores<F16, F16>(p, D, G, stream);
    else if (q_dtype == PKV_BF16) e = launch_scores<I8, BF16>(p, D, G, stream);
    else e = launch_scores<I8, F16>(p, D, G, stream);
    return done(e);
}

extern "C" pkv_status pkv_block_select(const float* scores, int32_t batch, int32_t num_kv_heads,
                                       int32_t max_blocks_per_seq, const int32_t* context_lens,
                                       int32_t keep_first, int32_t keep_last, int32_t budget,
                                       int32_t* block_lists, int32_t* list_lens,
                                       uint32_t* dev_status, cudaStream_t stream) {
    if (batch < 0 || num_kv_heads <= 0 || max_blocks_per_seq <= 0 ||
        max_blocks_per_seq > 0x7fffffff / kBlockSize || keep_first < 0 || keep_last < 0 ||
        budget <= 0 || (long long)keep_first + keep_last > budget)
        return PKV_ERR_INVALID_ARG;
    if (batch == 0) return PKV_OK;
    if (!scores || !context_lens || !block_lists || !list_lens) return PKV_ERR_INVALID_ARG;
    if (!aligned_to(scores, 4) || !aligned_to(context_lens, 4) || !aligned_to(block_lists, 4) ||
        !aligned_to(list_lens, 4) || !aligned_to(dev_status, 4))
        return PKV_ERR_INVALID_ARG;
    const long long rows = (long long)batch * num_kv_heads;
    if (rows > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
    SelectParams p;
    p.scores = scores; p.context_lens = context_lens; p.lists = block_lists; p.list_lens = list_lens;
    p.status = dev_status;
    p.hkv = num_kv_heads; p.mb = max_blocks_per_seq; p.budget = budget;
    p.keep_first = keep_first; p.keep_last = keep_last;
    p.cap = max_blocks_per_seq < choose::kKeepRow ? max_blocks_per_seq : choose::kKeepRow;
    const int threads = choose::threads_per_row(max_blocks_per_seq, rows);
    return done(threads == 1024  ? launch_select<1024>(p, int(rows), stream)
                : threads == 512 ? launch_select<512>(p, int(rows), stream)
                                 : launch_select<256>(p, int(rows), stream));
}
