// Multi-query attention with a sliding window: the tcgen05 kernel for long query runs
// over fp16, bf16 and INT8 caches (mq_wide.cu, mq_wide_i8.cu instantiate it).
//
// A CTA owns two tiles of 128 rows (query, head) of one (sequence, kv head) and walks
// the blocks that any of its rows sees in chunks of 128 tokens:
//   S = Q K^T   M = 128, N = 128, K = D, fp32 in tensor memory
//   softmax     a thread per row reads its S row twice, for the maximum and for P
//   O += P V    M = 128, N = D, K = 128; P in 16 bits from tensor memory, over the S that it
//               came from; O stays in tensor memory
// Tensor memory (512 columns): S of tile x at 128 x, O at 256 + 128 x. The MMAs of the one
// issuing thread run in order: P V of chunk c, then S of chunk c + 1 over the same columns,
// while the other tile's softmax works. Where only one tile holds queries, its even chunks
// take the first tile's place and its odd ones the second's, two states of the same rows
// that meet at the end.
//
// P over 16-bit caches comes in two parts of the cache's type (one bf16 part of a weight is
// off by 2^-9, as much as a bf16 output's rounding) and V as it is: a row's result then
// does not depend on the size of what other rows see. (bf16 V converted to fp16 for one
// part of P took 216 us for the prompt chunks below, and lost V's range to the largest
// value of its chunk.) INT8 codes of K and V enter as exact fp16 values, q in fp16 (bf16
// rows scaled into range by a power of two each); K's scale acts on S by block, V's on P,
// whose reference counts it (mq_scale_log in mq_split.cuh). P is one fp16 part there under a
// bf16 output, two under an fp16 one.
//
// Roles: warp 0 copies (TMA, 128-byte swizzle; INT8 as plain tiles), warp 1 issues the
// MMAs, warps 2-9 run the softmax and the epilogue, warps 10-13 convert INT8 K and V and
// zero the rows of 16-bit V that no row of the CTA may see (they may hold NaN).
//
// Why 128 tokens: a chunk of 64 pays the same waits for half the tokens, and two tiles' S
// and O of 128 columns each are what tensor memory holds.
//
// Measured (8 sequences of 2048 to 8192 tokens, their last 512 the queries, window 2048, 32 / 8
// heads, D = 128; floor of the products 72 us): 230 us over bf16 and fp16 caches, 236 over
// INT8 (302 with an fp16 q); D = 64 210, 214, 193 and 247. On the way: 64-token chunks
// (mq_tc.cuh's form with a window) 299; this form, with one part of P, with its column loops
// unrolled 582 (the code outran the instruction cache), in loops of 32 columns 233, with Q
// loaded while the copies start and the next columns read ahead 213. INT8, 6 runs of 3 to 301
// queries, window 1000, 16 / 8 heads: 85 us on mma.sync, 44 here. One tile, 64 sequences,
// window 4096, 8 kv heads (1.07 GB, 158 us at the copy rate): 280 us. 256 sequences of one
// query each under a max_q_len of 8192: 2071 us with a CTA for every pair that could be, 316 so.
// What bounds it: softmax and products of a chunk pair share a period and wait for one another
// (the products' pipe is 0.56 busy, the issue slots 0.42); the products alone are 3072 of its
// about 5400 cycles, the 320 KB that go through shared memory 2560 at least; then whole waves:
// 512 CTAs, one per SM, take 4 rounds of 152 for 3.37.
#pragma once

#include "mq_split.cuh"
#include "tc.cuh"

#include <algorithm>

namespace pkv {

// 16-bit caches: tensor maps; INT8: the cache and its scales.
using WideLaunch = cudaError_t (*)(const void* k_src, const void* v_src, const MqParams&, int,
                                   cudaStream_t);
WideLaunch wide_pick(pkv_dtype kv_dtype, int D, int G);          // fp16 / bf16: mq_wide.cu
WideLaunch wide_pick_i8(pkv_dtype q_dtype, int D, int G);        // mq_wide_i8.cu

namespace {

constexpr int kWideChunk = 128, kWideBlocks = kWideChunk / kBlockSize;
constexpr int kWideThreads = 448;
constexpr float kWideScaleUp = 128.f;   // INT8: P times V scales, up to 2^15 with the lazy rescale
// CTAs at most. One for every pair of tiles that max_q allows, of sequences with fewer queries
// too, would cost 6.3 ns for each that finds nothing to do.
constexpr int kWideGrid = 8 * 152;

// What the softmax needs to know of a chunk.
struct WideInfo {
    float ks[kWideBlocks], vs[kWideBlocks];   // INT8: scales of K, and of V by kWideScaleUp
    float lv[kWideBlocks];                    // mq_scale_log of V's
    int mask;                                 // blocks that are there
};

template <typename KV, typename QT, int D>
struct WideCfg {
    static constexpr bool kI8 = Elem<KV>::bytes == 1;
    static constexpr bool kTwo = !kI8 || std::is_same<QT, F16>::value;   // two parts of P
    using PT = typename std::conditional<std::is_same<KV, BF16>::value, BF16, F16>::type;   // of P and V
    // fp16 caches: P enters as 2^7 P, up to 2^15 with the lazy rescale
    static constexpr float kShift = std::is_same<KV, F16>::value ? 7.f : 0.f;
    static constexpr int NH = D / 64;                            // 64-column halves
    static constexpr int HALF = kWideChunk * 128;
    static constexpr int SLOT = NH * HALF;                       // K or V of a chunk in 16 bits
    static constexpr int QHALF = kTcRows * 128;
    static constexpr int QTILE = NH * QHALF;
    static constexpr int NK = kI8 ? 2 : 3, NV = 2;
    static constexpr int RAW = kI8 ? kWideChunk * D : 0;         // codes of K or V of a chunk
    static constexpr int OFF_K = 2 * QTILE, OFF_V = OFF_K + NK * SLOT, OFF_RAW = OFF_V + NV * SLOT;
    static constexpr int OFF_BAR = OFF_RAW + 2 * RAW;
    // barriers: k_full, k_empty, k_ready [NK]; v_full, v_empty, v_ready [NV]; raw_full,
    // raw_empty [K, V]; s_full, p_full, o_done [tile]; drain
    static constexpr int NBAR = 3 * NK + 3 * NV + 4 + 6 + 1;
    static constexpr int OFF_INFO = OFF_BAR + NBAR * 8;
    static constexpr int OFF_BLK = OFF_INFO + NV * int(sizeof(WideInfo));   // [2][8] physical blocks
    static constexpr int OFF_ROW = OFF_BLK + 2 * kWideBlocks * 4;           // INT8: 2^n of q's rows
    static constexpr int OFF_MISC = OFF_ROW + (kI8 ? 2 * kTcRows * 4 : 0);
    static constexpr int BYTES = OFF_MISC + 32 + 1024;
    static_assert(D == 64 || D == 128, "head_dim");
    static_assert(BYTES <= 232448 && OFF_RAW % 1024 == 0, "shared memory");
};

// 32 columns of this thread's TMEM lane; they may be used after wide_wait_ld.
__device__ __forceinline__ void wide_ld32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                   "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
                   "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
                   "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
                   "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr));
}
__device__ __forceinline__ void wide_wait_ld(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]),
                   "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]),
                   "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),
                   "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]) :: "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Two fp32 products in one operation.
__device__ __forceinline__ void wide_mul2(float& a, float& b, float f) {
    asm("{.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmul.rn.f32x2 x, x, y;\n\t"
        "mov.b64 {%0, %1}, x;}" : "+f"(a), "+f"(b) : "f"(f));
}

// The lowest n of 16 bits.
__device__ __forceinline__ uint32_t wide_below(int n) { return (1u << max(0, min(kBlockSize, n))) - 1u; }

// AND of a predicate over the 256 threads of the softmax.
__device__ __forceinline__ bool wide_all(bool x) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, 5, 256, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}" : "=r"(r) : "r"(uint32_t(x)) : "memory");
    return r != 0;
}

template <typename KV, typename QT, int D, int G>
__global__ void __launch_bounds__(kWideThreads, 1)
mq_wide_kernel(const __grid_constant__ MqSrc<KV> ksrc, const __grid_constant__ MqSrc<KV> vsrc, const MqParams p) {
    using C = WideCfg<KV, QT, D>;
    constexpr bool kI8 = C::kI8;
    using PT = typename C::PT;
    constexpr int NK = C::NK, NV = C::NV, NH = C::NH, NB = kWideBlocks;
    constexpr int QPT = kTcRows / G;                       // queries per tile
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t *k_full = bars, *k_empty = bars + NK, *k_ready = bars + 2 * NK;
    uint64_t *v_full = bars + 3 * NK, *v_empty = v_full + NV, *v_ready = v_full + 2 * NV;
    uint64_t *raw_full = v_full + 3 * NV, *raw_empty = raw_full + 2;
    uint64_t *s_full = raw_full + 4, *p_full = s_full + 2, *o_done = s_full + 4, *drain = s_full + 6;
    WideInfo* infos = reinterpret_cast<WideInfo*>(smem + C::OFF_INFO);
    int* sblk = reinterpret_cast<int*>(smem + C::OFF_BLK);
    float* srow = reinterpret_cast<float*>(smem + C::OFF_ROW);
    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);   // TMEM, abort, -, unit
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    griddep_wait();
    griddep_launch_dependents();
    // unit: (sequence b, kv head, tile pair u), later pairs first. Grids of one CTA for
    // every pair that max_q allows find theirs by division; smaller ones (wide_launch)
    // count the pairs that there are, each thread those of a run of sequences, and walk
    // them.
    const int tpair = (p.tmax + 1) / 2;
    const long long all_pairs = (long long)p.batch * p.hkv * tpair;
    const bool direct = all_pairs <= gridDim.x;
    int total = int(all_pairs), mine0 = 0, mine = 0;       // compact: this thread's units
    const int run = (p.batch + kWideThreads - 1) / kWideThreads;
    const int seq0 = min(p.batch, int(threadIdx.x) * run), seq9 = min(p.batch, seq0 + run);
    auto pairs_of = [&](int b, bool flag) {
        int n, L;
        bool bad;
        seq_shape_raw(p.cu_q, p.context_lens, b, p.mb, p.max_q, n, L, bad);
        if (bad && flag) flag_status(p.status, PKV_DEV_BAD_LENGTH);
        return (n * G + 2 * kTcRows - 1) / (2 * kTcRows);
    };
    if (!direct) {
        for (int b = seq0; b < seq9; ++b) mine += p.hkv * pairs_of(b, blockIdx.x == 0);
        int* sums = reinterpret_cast<int*>(smem);          // of the warps
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) sums[warp] = inc;
        __syncthreads();
        total = 0;
        for (int w = 0; w < kWideThreads / 32; ++w) {
            if (w == warp) mine0 = total + inc - mine;
            total += sums[w];
        }
    }
    uint32_t tmem = 0u;
    bool allocated = false;
    for (int unit = blockIdx.x; unit < total; unit += gridDim.x) {
    int b, kvh, u;
    if (direct) {
        u = tpair - 1 - unit % tpair;
        kvh = unit / tpair % p.hkv;
        b = unit / tpair / p.hkv;
    } else {
        if (unit >= mine0 && unit < mine0 + mine) {
            int at = mine0, x = seq0, pairs = 0;
            for (;; ++x) {
                pairs = pairs_of(x, false);
                if (unit < at + pairs * p.hkv || x + 1 == seq9) break;
                at += pairs * p.hkv;
            }
            misc[3] = x;
            misc[4] = (unit - at) / pairs;
            misc[5] = pairs - 1 - (unit - at) % pairs;
        }
        __syncthreads();
        b = misc[3];
        kvh = misc[4];
        u = misc[5];
    }
    int n, L;
    bool bad;
    seq_shape_raw(p.cu_q, p.context_lens, b, p.mb, p.max_q, n, L, bad);
    if (bad && threadIdx.x == 0 && kvh == 0 && u == 0) flag_status(p.status, PKV_DEV_BAD_LENGTH);
    const int q00 = 2 * u * QPT;                           // first query of tile 0
    if (q00 >= n) break;                                   // direct: the CTA's only unit, nothing allocated
    const bool two = q00 + QPT < n;                        // tile 1 holds queries too
    const int cu = p.cu_q[b];
    const int q_last = min(n, q00 + (two ? 2 : 1) * QPT) - 1;
    const MqShown see = mq_shown(L - n + q00, p.window, p.sinks);
    const int nblk = (L - n + q_last) / kBlockSize + 1 - see.skip;   // blocks that any row sees
    const int nch = (nblk + NB - 1) / NB;
    auto block_at = [&](int j) { return j >= see.lead ? j + see.skip : j; };

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NBAR; ++i) mbar_init(smem_addr(&bars[i]), 1);
        for (int i = 0; i < NK; ++i) mbar_init(smem_addr(&k_ready[i]), 4);
        for (int i = 0; i < NV; ++i) mbar_init(smem_addr(&v_ready[i]), 4);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&raw_empty[i]), 4);
            mbar_init(smem_addr(&p_full[i]), 4);
        }
        fence_mbar_init();
        misc[1] = 0u;
    }
    if (warp == 1 && !allocated) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_addr((const void*)(misc + 0))), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    tmem = misc[0];
    allocated = true;

    // both Q tiles (query q00 + R / G, head R % G for R in 0 .. 255), zero past the
    // sequence, 128-byte-swizzled K-major, by all warps but the producer, which is off
    // already. 16-byte pieces; a row's D / 8 lie in adjacent lanes, which is how INT8
    // finds its maximum.
    if (warp != 0) {
        constexpr int PPR = D / 8, LOADERS = kWideThreads - 32, PIECES = 2 * kTcRows * PPR;
        constexpr int N = (PIECES + LOADERS - 1) / LOADERS;
        static_assert(PIECES % LOADERS % 32 == 0 && 32 % PPR == 0, "whole warps and rows");
        uint4 v[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = int(threadIdx.x) - 32 + k * LOADERS, R = i / PPR, qi = q00 + R / G;
            v[k] = make_uint4(0u, 0u, 0u, 0u);
            if (i < PIECES && qi < n)
                v[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                            ((long long)(cu + qi) * p.hq + kvh * G + R % G) * D + i % PPR * 8));
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = int(threadIdx.x) - 32 + k * LOADERS, R = i / PPR, c16 = i % PPR;
            if (i >= PIECES) break;                        // whole warps
            if constexpr (kI8) {
                uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
                float amax = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = unpack2(QT{}, w[j]);
                    amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
#pragma unroll
                for (int o = 1; o < PPR; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
                const float2 fit = std::is_same<QT, BF16>::value ? fit_half(amax) : make_float2(1.f, 1.f);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = unpack2(QT{}, w[j]);
                    w[j] = pack2<F16>(f.x * fit.x, f.y * fit.x);
                }
                v[k] = make_uint4(w[0], w[1], w[2], w[3]);
                if (c16 == 0) srow[R] = fit.y;
            }
            const int half = c16 / 8, c = c16 % 8, r = R % kTcRows;
            *reinterpret_cast<uint4*>(smem + R / kTcRows * C::QTILE + half * C::QHALF + r * 128 + ((c ^ (r & 7)) << 4)) = v[k];
        }
        fence_proxy_async_smem();
        asm volatile("barrier.cta.sync 4, %0;" :: "n"(LOADERS) : "memory");
    }

    auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t role_bit) -> bool {
        if (misc[1]) return false;
        const bool ok = mbar_wait_bounded(smem_addr(bar), parity & 1u, p.wait_ns);
        if (!ok) {
            misc[1] = 1u;
            flag_status(p.status, PKV_DEV_TIMEOUT | role_bit);
        }
        return ok;
    };
    // the slot of chunk c is free: chunk c - slots has left it
    auto wait_free = [&](uint64_t* empty, int slots, int c, uint32_t role_bit) {
        return c < slots || wait(&empty[c % slots], c / slots - 1, role_bit);
    };

    if (warp == 0) {
        // ------------------------------------------------------ producer ---
        // lane jj < 8 looks up and copies block jj of a chunk, the table one chunk ahead
        auto lookup = [&](int c) {
            const int j = c * NB + lane;
            return lane < NB && j < nblk ? __ldg(p.block_tables + (long long)b * p.mb + block_at(j)) : -1;
        };
        int next = lookup(0), k_issued = 0, v_issued = 0;
        for (int c = 0; c < nch; ++c) {
            int blk = next;
            next = c + 1 < nch ? lookup(c + 1) : -1;
            const bool listed = lane < NB && c * NB + lane < nblk;
            if (listed && unsigned(blk) >= unsigned(p.num_blocks)) flag_status(p.status, PKV_DEV_BAD_BLOCK);
            if (!listed || unsigned(blk) >= unsigned(p.num_blocks)) blk = -1;
            const int count = __popc(__ballot_sync(kFull, blk >= 0));
            const uint32_t extra = (c == 0 && unit == p.stall_cta) ? 16u : 0u;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                uint64_t* full = kI8 ? &raw_full[kv] : kv ? &v_full[c % NV] : &k_full[c % NK];
                const bool ok = kI8 ? (c == 0 || wait(&raw_empty[kv], c - 1, 0x400u))
                                    : kv ? wait_free(v_empty, NV, c, 0x400u) : wait_free(k_empty, NK, c, 0x400u);
                if (!__all_sync(kFull, ok)) goto produced;
                const uint32_t bar = smem_addr(full);
                if (kv && lane < NB) sblk[(c & 1) * NB + lane] = blk;
                __syncwarp();
                if (lane == 0) {
                    const uint32_t tx = count * (kI8 ? kBlockSize * D : NH * kBlockSize * 128) + (kv ? 0u : extra);
                    if (tx) mbar_arrive_expect_tx(bar, tx);
                    else mbar_arrive(bar);
                }
                __syncwarp();
                if (blk >= 0) {
                    if constexpr (kI8) {
                        const MqI8Src& src = kv ? vsrc : ksrc;
                        bulk_g2s(smem_addr(smem + C::OFF_RAW + kv * C::RAW + lane * kBlockSize * D),
                                 static_cast<const char*>(src.cache) + ((long long)blk * p.hkv + kvh) * (kBlockSize * D),
                                 kBlockSize * D, bar);
                    } else {
                        const int y = (blk * p.hkv + kvh) * kBlockSize;
                        unsigned char* dst = smem + (kv ? C::OFF_V + c % NV * C::SLOT : C::OFF_K + c % NK * C::SLOT) +
                                             lane * kBlockSize * 128;
#pragma unroll
                        for (int h = 0; h < NH; ++h)
                            tma_load_2d(smem_addr(dst + h * C::HALF), kv ? &vsrc : &ksrc, 64 * h, y, bar);
                    }
                }
                if (kv) v_issued = c + 1;
                else k_issued = c + 1;
            }
        }
    produced:
        // The CTA exits with no copy in flight, after an abort too: the last of each slot
        // land (bounded).
        if (lane == 0) {
            if constexpr (kI8) {
                if (k_issued) mbar_wait_bounded(smem_addr(&raw_full[0]), (k_issued - 1) & 1, p.wait_ns);
                if (v_issued) mbar_wait_bounded(smem_addr(&raw_full[1]), (v_issued - 1) & 1, p.wait_ns);
            } else {
                for (int c = max(0, k_issued - NK); c < k_issued; ++c)
                    mbar_wait_bounded(smem_addr(&k_full[c % NK]), (c / NK) & 1, p.wait_ns);
                for (int c = max(0, v_issued - NV); c < v_issued; ++c)
                    mbar_wait_bounded(smem_addr(&v_full[c % NV]), (c / NV) & 1, p.wait_ns);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer ---
        if (lane == 0) {
            const uint32_t id_s = tc_idesc(std::is_same<KV, BF16>::value ? 1u : 0u, 0, kWideChunk, kTcRows);
            const uint32_t id_o = tc_idesc(std::is_same<typename C::PT, BF16>::value ? 1u : 0u, 1, D, kTcRows);
            const uint64_t dq0 = tc_desc(smem_addr(smem), 16, 1024);
            const uint64_t dk0 = tc_desc(smem_addr(smem + C::OFF_K), 16, 1024);
            const uint64_t dv0 = tc_desc(smem_addr(smem + C::OFF_V), C::HALF, 1024);
            uint64_t* k_there = kI8 ? k_ready : k_full;
            auto issue_s = [&](int c, int x, int xq) {
                const uint64_t dq = dq0 + uint64_t((xq * C::QTILE) >> 4);
                const uint64_t dk = dk0 + uint64_t((c % NK) * (C::SLOT >> 4));
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    tc_mma(tmem + x * kWideChunk, dq + (((kk / 4) * C::QHALF + (kk % 4) * 32) >> 4),
                           dk + (((kk / 4) * C::HALF + (kk % 4) * 32) >> 4), id_s, kk > 0);
                tc_commit(smem_addr(&s_full[x]));
            };
            auto issue_pv = [&](int c, int x, bool more) {
                const uint64_t dv = dv0 + uint64_t((c % NV) * (C::SLOT >> 4));
                const uint32_t tp = tmem + x * kWideChunk, to = tmem + 2 * kWideChunk + x * 128;
#pragma unroll
                for (int part = 0; part < (C::kTwo ? 2 : 1); ++part)
#pragma unroll
                    for (int kk = 0; kk < kWideChunk / 16; ++kk)
                        tc_mma_ts(to, tp + (kk / 2) * 32 + (kk & 1) * 8 + part * 16, dv + uint64_t((kk * 16 * 128) >> 4), id_o,
                                  (more || part > 0 || kk > 0) ? 1u : 0u);
            };
            auto k_in = [&](int c) {
                const bool in = wait(&k_there[c % NK], c / NK, 0x800u);
                tc_fence_after();
                return in;
            };
            auto v_in = [&](int c, int x, int phase) {
                const bool in = wait(&v_ready[c % NV], c / NV, 0x800u) && wait(&p_full[x], phase, 0x800u);
                tc_fence_after();
                return in;
            };
            auto k_out = [&](int c) { tc_commit(smem_addr(&k_empty[c % NK])); };
            auto v_out = [&](int c) { tc_commit(smem_addr(&v_empty[c % NV])); };
            bool ok = true;
            if (two) {
                if ((ok = k_in(0))) {
                    issue_s(0, 0, 0);
                    issue_s(0, 1, 1);
                    k_out(0);
                }
                for (int c = 0; c < nch && ok; ++c) {
                    const bool more = c + 1 < nch;
                    if (!(ok = v_in(c, 0, c))) break;
                    issue_pv(c, 0, c > 0);
                    if (more) {
                        if (!(ok = k_in(c + 1))) break;
                        issue_s(c + 1, 0, 0);
                    }
                    if (!(ok = wait(&p_full[1], c, 0x800u))) break;
                    tc_fence_after();
                    issue_pv(c, 1, c > 0);
                    v_out(c);
                    if (more) {
                        issue_s(c + 1, 1, 1);
                        k_out(c + 1);
                    }
                }
            } else {
                for (int c = 0; c < min(2, nch) && ok; ++c) {
                    if (!(ok = k_in(c))) break;
                    issue_s(c, c, 0);
                    k_out(c);
                }
                for (int c = 0; c < nch && ok; ++c) {
                    if (!(ok = v_in(c, c & 1, c >> 1))) break;
                    issue_pv(c, c & 1, c > 1);
                    v_out(c);
                    if (c + 2 < nch) {
                        if (!(ok = k_in(c + 2))) break;
                        issue_s(c + 2, c & 1, 0);
                        k_out(c + 2);
                    }
                }
            }
            if (ok) {
                tc_commit(smem_addr(&o_done[0]));
                tc_commit(smem_addr(&o_done[1]));
            }
            tc_commit(smem_addr(&drain[0]));
            mbar_wait_bounded(smem_addr(&drain[0]), 0, 2000000000ull);
            if (ok && unit + (long long)gridDim.x < total) {   // every arrival has come before the next unit
                for (int c = max(0, nch - NK); c < nch; ++c) wait(&k_empty[c % NK], c / NK, 0x800u);
                for (int c = max(0, nch - NV); c < nch; ++c) wait(&v_empty[c % NV], c / NV, 0x800u);
                for (int x = 0; x < 2; ++x) wait(&o_done[x], 0, 0x800u);
            }
        }
    } else if (warp >= 10) {
        // ---------------------------------------------------- converters ---
        const int t = int(threadIdx.x) - 320;
        bool ok = true;
        for (int c = 0; c < nch; ++c) {
            unsigned char* kd = smem + C::OFF_K + c % NK * C::SLOT;
            unsigned char* vd = smem + C::OFF_V + c % NV * C::SLOT;
            WideInfo* info = infos + c % NV;
            if constexpr (kI8) {
                // 16 codes of a token -> two 16-byte pieces of the swizzled tile
                auto expand = [&](const unsigned char* raw, unsigned char* dst) {
                    constexpr int PIECES = D / 16;
#pragma unroll 4
                    for (int i = t; i < kWideChunk * PIECES; i += 128) {
                        const int tok = i / PIECES, pc = i % PIECES;
                        const uint4 x = *reinterpret_cast<const uint4*>(raw + tok * D + pc * 16);
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                        uint32_t o[8];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t y = w[k] ^ 0x80808080u;
                            const uint32_t h0 = i8x2_biased_h2(y, 0x4140), h1 = i8x2_biased_h2(y, 0x4342);
                            const __half2 bias = __half2half2(__ushort_as_half(0x6480));     // 1152
                            const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&h0), bias);
                            const __half2 z = __hsub2(*reinterpret_cast<const __half2*>(&h1), bias);
                            o[2 * k] = *reinterpret_cast<const uint32_t*>(&a);
                            o[2 * k + 1] = *reinterpret_cast<const uint32_t*>(&z);
                        }
                        unsigned char* row = dst + (pc / 4) * C::HALF + tok * 128;
                        const int c16 = 2 * (pc % 4), sw = tok & 7;
                        *reinterpret_cast<uint4*>(row + ((c16 ^ sw) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4*>(row + (((c16 + 1) ^ sw) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                };
                ok = wait(&raw_full[0], c, 0x2000u) && wait_free(k_empty, NK, c, 0x2000u);
                if (!__all_sync(kFull, ok)) break;
                expand(smem + C::OFF_RAW, kd);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_addr(&raw_empty[0]));
                    mbar_arrive(smem_addr(&k_ready[c % NK]));
                }
                ok = wait(&raw_full[1], c, 0x2000u) && wait_free(v_empty, NV, c, 0x2000u);
                if (!__all_sync(kFull, ok)) break;
                // scales: lanes 0-7 V's, 8-15 K's
                const int blk = lane < 2 * NB ? sblk[(c & 1) * NB + lane % NB] : -1;
                float sc = 0.f;
                if (blk >= 0) sc = __ldg((lane < NB ? vsrc.scales : ksrc.scales) + (long long)blk * p.hkv + kvh);
                const int mask = int(__ballot_sync(kFull, blk >= 0) & 0xffu);
                expand(smem + C::OFF_RAW + C::RAW, vd);
                if (t < 2 * NB) {
                    // (K codes of 0 by any scale, so that -inf stays -inf)
                    if (t < NB) {
                        info->vs[t] = sc * kWideScaleUp;
                        info->lv[t] = mq_scale_log(sc);
                    } else {
                        info->ks[t - NB] = sc != 0.f ? sc : 1e-38f;
                    }
                    if (t == 0) info->mask = mask;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_addr(&raw_empty[1]));
                    mbar_arrive(smem_addr(&v_ready[c % NV]));
                }
            } else {
                ok = wait(&v_full[c % NV], c / NV, 0x2000u);
                if (!__all_sync(kFull, ok)) break;
                const int blk = lane < NB ? sblk[(c & 1) * NB + lane] : -1;
                const int mask = int(__ballot_sync(kFull, blk >= 0) & 0xffu);
                // piece i of the thread: row t / 8 of block i % 8, as it lies
                auto hidden = [&](int i) {
                    const int tok = kBlockSize * block_at(c * NB + i % NB) + t / 8;
                    return !((mask >> (i % NB)) & 1) || tok >= L || (tok >= see.sinks && tok < see.first);
                };
                // whole: every row of the chunk may be seen by some row (uniform)
                const int t0 = kBlockSize * block_at(c * NB), t9 = kBlockSize * (block_at(c * NB + NB - 1) + 1);
                const bool whole = mask == 0xff && t9 <= L && (t0 >= see.first || t9 <= see.sinks);
                uint4* at = reinterpret_cast<uint4*>(vd) + t;
                if (!whole)
                    for (int i = 0; i < NH * NB; ++i)
                        if (hidden(i)) at[128 * i] = make_uint4(0u, 0u, 0u, 0u);
                if (t == 0) info->mask = mask;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&v_ready[c % NV]));
            }
        }
    } else {
        // -------------------------------------- softmax + epilogue, per tile ---
        const int x = (warp - 2) >> 2;                        // tile, or parity of the chunks
        {
            const int r = 32 * (warp & 3) + lane;             // TMEM lane = row of the tile
            const uint32_t lane_addr = uint32_t(32 * (warp & 3)) << 16;
            const uint32_t tm_s = tmem + x * kWideChunk + lane_addr;
            const uint32_t tm_o = tmem + 2 * kWideChunk + x * 128 + lane_addr;
            const int qi = q00 + (two ? x * QPT : 0) + r / G;
            const bool rv = qi < n, none = !__any_sync(kFull, rv);
            const int pos = L - n + qi;
            const float qs = kI8 ? p.qscale * srow[two ? x * kTcRows + r : r] : p.qscale;
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            const int start = two ? 0 : x, step = two ? 1 : 2;
            for (int c = start, phase = 0; c < nch; c += step, ++phase) {
                // S of chunk c is there, and with it (in order) P V of the chunk before
                ok = wait(&s_full[x], phase, 0x1000u) && wait(&v_ready[c % NV], c / NV, 0x1000u);
                if (!__all_sync(kFull, ok)) {
                    ok = false;
                    break;
                }
                if (none) {                                   // no query in the warp's rows: P may be anything
                    if (lane == 0) mbar_arrive(smem_addr(&p_full[x]));
                    continue;
                }
                tc_fence_after();
                const WideInfo* info = infos + c % NV;
                const int mask = info->mask;
                const int t0 = kBlockSize * block_at(c * NB), t9 = kBlockSize * (block_at(c * NB + NB - 1) + 1) - 1;
                // warp-uniform: every row sees every token, and its largest score is that
                // of its largest S
                // (rows past the last query hold zeros)
                const bool plain = __all_sync(kFull, mask == 0xff && p.qscale > 0.f &&
                                                     (!rv || (pos >= t9 && (p.window == 0 || t0 > pos - p.window || t9 < p.sinks))));
                // bits of a block's tokens that the row sees
                auto shown = [&](int j) -> uint32_t {
                    const int at = kBlockSize * block_at(c * NB + j);
                    if (!rv || !((mask >> j) & 1)) return 0u;
                    const int from = p.window == 0 ? 0 : pos - p.window + 1;
                    return wide_below(pos + 1 - at) & (wide_below(p.sinks - at) | ~wide_below(from - at));
                };
                // ---- the row's maximum, 32 columns at a time, the next being read meanwhile.
                // (Loops, not straight code: the 128 columns of two passes, plain and masked,
                // outran the instruction cache: 582 us for what took 233 so.) Masked columns
                // go back as scores in log2 units, hidden ones -inf.
                float mx = -INFINITY;
                auto take_max = [&](uint32_t (&w)[32], int q) {
                    if (!plain) {
                        const uint32_t vis = shown(2 * q) | shown(2 * q + 1) << 16;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            w[i] = __float_as_uint((vis >> i & 1u) ? __uint_as_float(w[i]) * qs : -INFINITY);
                        tc_st16(tm_s + 32 * q, w);
                        tc_st16(tm_s + 32 * q + 16, w + 16);
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float bm = __uint_as_float(w[16 * j]), bn = __uint_as_float(w[16 * j + 1]);
#pragma unroll
                        for (int i = 2; i < 14; i += 4) {
                            bm = max3(bm, __uint_as_float(w[16 * j + i]), __uint_as_float(w[16 * j + i + 1]));
                            bn = max3(bn, __uint_as_float(w[16 * j + i + 2]), __uint_as_float(w[16 * j + i + 3]));
                        }
                        bm = max3(bm, bn, fmaxf(__uint_as_float(w[16 * j + 14]), __uint_as_float(w[16 * j + 15])));
                        if (plain) bm *= qs;
                        if constexpr (kI8) bm = fmaf(bm, info->ks[2 * q + j], info->lv[2 * q + j]);
                        mx = fmaxf(mx, bm);
                    }
                };
                uint32_t sa[32], sb[32];
                wide_ld32(tm_s, sa);
                wide_wait_ld(sa);
#pragma unroll 1
                for (int q = 0; q < 4; q += 2) {
                    wide_ld32(tm_s + 32 * (q + 1), sb);
                    take_max(sa, q);
                    wide_wait_ld(sb);
                    if (q == 0) wide_ld32(tm_s + 64, sa);
                    take_max(sb, q + 1);
                    if (q == 0) wide_wait_ld(sa);
                }
                if (!plain) tc_wait_st();
                const bool grow = mx > m + kTcLazy || (m == -INFINITY && mx > -INFINITY);
                float a = 1.f;
                if (grow) {
                    if (m > -INFINITY) a = fast_exp2(m - mx);
                    l *= a;
                    m = mx;
                }
                if (c > start && __any_sync(kFull, a != 1.f)) {
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        float o[32];
                        tc_ld32(tm_o + c0, o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] *= a;
                        tc_st32(tm_o + c0, o);
                    }
                }
                // ---- P over the S that it came from: of 32 columns the first 16 take P's first
                // part, the others its second. (16-bit caches: l counts what P enters as)
                const float nm = (m == -INFINITY ? 0.f : -m) + C::kShift, qp = plain ? qs : 1.f;
                auto put_p = [&](uint32_t (&w)[32], int q) {
                    uint32_t hw[16];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float kq = kI8 ? qp * info->ks[2 * q + j] : qp;
                        const float f = kI8 ? info->vs[2 * q + j] : 1.f;
                        float s0 = 0.f, s1 = 0.f;
#pragma unroll
                        for (int i = 8 * j; i < 8 * j + 8; ++i) {
                            float x0 = fast_exp2(fmaf(__uint_as_float(w[2 * i]), kq, nm));
                            float x1 = fast_exp2(fmaf(__uint_as_float(w[2 * i + 1]), kq, nm));
                            s0 += x0;
                            s1 += x1;
                            if constexpr (kI8) wide_mul2(x0, x1, f);
                            hw[i] = pack2<PT>(x0, x1);
                            if constexpr (C::kTwo) {
                                const float2 rr = unpack2(PT{}, hw[i]);
                                w[i] = pack2<PT>(x0 - rr.x, x1 - rr.y);
                            }
                        }
                        l += s0 + s1;
                    }
                    tc_st16(tm_s + 32 * q, hw);
                    if constexpr (C::kTwo) tc_st16(tm_s + 32 * q + 16, w);
                };
                wide_ld32(tm_s, sa);
                wide_wait_ld(sa);
#pragma unroll 1
                for (int q = 0; q < 4; q += 2) {
                    wide_ld32(tm_s + 32 * (q + 1), sb);
                    put_p(sa, q);
                    wide_wait_ld(sb);
                    if (q == 0) wide_ld32(tm_s + 64, sa);
                    put_p(sb, q + 1);
                    if (q == 0) wide_wait_ld(sa);
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&p_full[x]));
            }
            if (ok) ok = __all_sync(kFull, wait(&o_done[x], 0, 0x1000u));   // all products, of both tiles
            float2* states = reinterpret_cast<float2*>(smem + C::QTILE);
            if (!two) {                                       // all 8 warps come here, whatever happened
                states[x * kTcRows + r] = make_float2(m, l);
                ok = wide_all(ok);
            }
            if (ok) {
                tc_fence_after();
                uint16_t* dst = static_cast<uint16_t*>(p.out) + ((long long)(cu + qi) * p.hq + kvh * G + r % G) * D;
                // One tile: the states of the even and odd chunks meet, and each half of the warps
                // writes half of the columns.
                float sum = l, g0 = 1.f, g1 = 0.f;
                const bool join = !two && nch > 1;            // else no odd chunk
                uint32_t from = tm_o;
                if (!two) {
                    const float2 s0 = states[r], s1 = states[kTcRows + r];
                    from = tmem + 2 * kWideChunk + lane_addr;
                    sum = s0.y;
                    if (join) {
                        const float top = fmaxf(s0.x, s1.x);
                        const float a0 = top == -INFINITY ? 1.f : fast_exp2(s0.x - top);
                        const float a1 = top == -INFINITY ? 1.f : fast_exp2(s1.x - top);
                        sum = fmaf(s0.y, a0, s1.y * a1);
                        g0 = a0;
                        g1 = a1;
                    }
                }
                const float inv = sum != 0.f ? (kI8 ? 1.f / kWideScaleUp : 1.f) / sum : 0.f;
                const int cols = two ? D : D / 2;
#pragma unroll 1
                for (int c0 = two ? 0 : x * cols, c9 = c0 + cols; c0 < c9; c0 += 32) {
                    float o[32];
                    tc_ld32(from + c0, o);
                    if (join) {
                        float o1[32];
                        tc_ld32(from + 128 + c0, o1);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = fmaf(o1[i], g1, o[i] * g0);
                    }
                    if (rv) {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) w[i] = pack2<QT>(o[2 * i] * inv, o[2 * i + 1] * inv);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            reinterpret_cast<uint4*>(dst + c0)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                    }
                    __syncwarp();
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (misc[1]) break;
    if (threadIdx.x == 0 && unit + (long long)gridDim.x < total)
        for (int i = 0; i < C::NBAR; ++i)
            asm volatile("mbarrier.inval.shared::cta.b64 [%0];" :: "r"(smem_addr(&bars[i])) : "memory");
    }
    if (warp == 1 && allocated)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(512));
}

// ------------------------------------------------------------------- host ---
template <typename KV, typename QT, int D, int G>
cudaError_t wide_launch(const void* k, const void* v, const MqParams& p, int grid, cudaStream_t st) {
    const int smem = WideCfg<KV, QT, D>::BYTES;
    const auto kernel = mq_wide_kernel<KV, QT, D, G>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(std::min(grid, kWideGrid)), dim3(kWideThreads), size_t(smem), st,
                      *static_cast<const MqSrc<KV>*>(k), *static_cast<const MqSrc<KV>*>(v), p);
}
template <typename KV, typename QT, int D>
WideLaunch wide_pick_g(int G) {
    switch (G) {
        case 1: return wide_launch<KV, QT, D, 1>;
        case 2: return wide_launch<KV, QT, D, 2>;
        case 4: return wide_launch<KV, QT, D, 4>;
        case 8: return wide_launch<KV, QT, D, 8>;
    }
    return nullptr;
}
template <typename KV, typename QT>
WideLaunch wide_pick_d(int D, int G) {
    return D == 128 ? wide_pick_g<KV, QT, 128>(G) : D == 64 ? wide_pick_g<KV, QT, 64>(G) : nullptr;
}

}  // namespace
}  // namespace pkv
