// Decode attention over chosen blocks, and decode attention that also reports
// each token's weight: one split kernel and one join kernel in two modes.
//
//   kList  the tokens of (sequence b, kv head) are the 16-token blocks that
//          its list names; out = softmax(scale q K^T) V over them.
//   kMass  all tokens of the sequence; besides out, every token's weights
//          p_ht = exp(s_ht - M_h) / l_h, summed over the head group, are added
//          to an accumulator.
//
// Mathematics: one pass over K and V with a running maximum m and sum l of
// the exponentials per head, in base 2; pieces (m, l, o) merge as
// sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i. A weight needs the final M
// and l, which a single pass has only at its end: kMass keeps the scores in
// the workspace (4 bytes per head and token, 6 % of the bytes that K and V
// cost at 4 heads per group in 16 bits, against 50 % for reading K again)
// and the join kernel turns them into weights.
//
// Both are bound by memory bandwidth. The unit of work is 8 KB of K and V of
// one kv head (1, 2 or 4 blocks). The units of the batch, in the order
// (sequence, kv head, entry), are cut into equal contiguous ranges, one per
// worker warp, so that ragged batches stay balanced. A warp feeds itself: its
// lanes issue one bulk copy for each K and V tile of a unit into two stages,
// with list and table entries fetched 32 units ahead. Scores and P V run on
// mma.sync m16n8k16 with the group's heads in the N columns, so a tile is read
// once for all heads of the group.
//
// Short calls take another form of the same kernel, a CTA or a cluster of them
// per segment that finishes it alone (ctas_per_segment).
//
// Measured (g = 4, D = 128, bf16): 256 sequences of 128 to 4096 tokens with
// weights 379 us, 2.26 GB (6.0 TB/s; with the scores 2.39 GB, 6.3 TB/s, 0.94 of
// the copy rate); 128 listed blocks of 64 sequences 88 us for 541 MB in the
// split (6.1 TB/s) and 4 in the join. INT8: 256 listed blocks of 48 sequences
// (g = 8, D = 128) 42 us for 203 MB, of which 5 pass before the first data and 5
// between the first and the last worker's end; 64 sequences with weights (g =
// 1, D = 64) 126 us for 580 MB (121 over the same inputs again), with 0.54 of the
// issue slots and 0.64 of DRAM in use: 12 warps per SM do not hide the chain of a
// unit. One sequence of 1023 tokens with weights, 8 kv heads: 7.8 us by clusters of 8
// CTAs, 14.1 split and joined.
#pragma once

#include "common.cuh"

#include <algorithm>
#include <atomic>

namespace pkv {
namespace ctx {

enum Mode { kList = 0, kMass = 1 };

constexpr int kOneWarps = 8;                         // warps per CTA where CTAs finish a segment
constexpr int kMaxWarps = 6;                         // worker warps per CTA otherwise, at most
constexpr uint64_t kWaitLimitNs = 4000000000ull;     // 4 s per bounded wait
constexpr uint64_t kDrainLimitNs = 100000000ull;     // 100 ms when draining
constexpr int kMaxBatch = 8192;
constexpr float kLog2e = 1.4426950408889634f;

__host__ __device__ constexpr int align_up(int x, int a) { return (x + a - 1) / a * a; }

// Unit prefix over the sequences in shared memory: exact up to kPrefixEntries
// sequences, beyond that every stride-th entry (a lookup then walks at most
// stride sequences), so that its size does not grow with the batch.
constexpr int kPrefixEntries = 256;
constexpr int kPrefixBytes = align_up(4 * kMaxWarps + 4 * (kPrefixEntries + 1), 128);

template <typename KV, typename QT, int D, int G>
struct Cfg {
    static constexpr bool kI8 = Elem<KV>::bytes == 1;
    static constexpr int ROW = D * Elem<KV>::bytes;               // bytes of one token row
    static constexpr int TILE = kBlockSize * ROW;
    // A unit is 8 KB of K and V whatever the type and head_dim (1, 2 or 4
    // blocks), so that its fixed costs (wait, copy issue, softmax shuffles)
    // are shared by the same bytes.
    static constexpr int STAGE = 8192;                            // K tiles [UB], V tiles [UB]
    static constexpr int UB = STAGE / (2 * TILE);                 // blocks per unit
    static constexpr int NS = 2;                                  // stages per warp
    static constexpr int OFF_BAR = NS * STAGE;
    static constexpr int OFF_META = align_up(OFF_BAR + NS * 8, 16);    // int4 per stage
    static constexpr int OFF_SCL = OFF_META + NS * 16;                 // float2 per stage, block
    static constexpr int OFF_P = align_up(OFF_SCL + NS * UB * 8, 16);  // P[head][token], fp32
    static constexpr int PS = UB * kBlockSize + 8;                // + 8: rows of P in other banks
    static constexpr int WARP_BYTES = align_up(OFF_P + PS * G * 4, 128);
    // 12 worker warps per SM for INT8, whose arithmetic needs them, in 2 CTAs
    // of 6; CTAs of 4 for 16-bit caches.
    static constexpr int WARPS = kI8 ? 6 : 4;
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int MIN_CTAS = kI8 ? 2 : 3;                  // registers per thread: 170
    static constexpr int SMEM = kPrefixBytes + WARPS * WARP_BYTES;
    static constexpr int SMEM_ONE = kPrefixBytes + kOneWarps * WARP_BYTES;
    // mbarrier arrivals of a stage: the byte count, and for INT8 one per scale
    static constexpr int ARRIVALS = kI8 ? 1 + 2 * UB : 1;
    // P in two 16-bit parts, hi = rn(P) and lo = rn(P - hi): for 16-bit caches,
    // and for INT8 ones whose output is fp16 (one fp16 part is off by 2^-11 of
    // the weight, as much as the output's own rounding; a bf16 output, which
    // rounds by 2^-8, hides it: 0.0017 against 64 bits with one part and with
    // two, which take 2 to 8 % longer, 58.4 instead of 56.3 us for 48 lists of
    // 256 blocks at g = 8).
    static constexpr bool kTwoParts = !kI8 || std::is_same<QT, F16>::value;
    // q of a bf16 call over INT8 codes is scaled into fp16's range
    static constexpr bool kFit = kI8 && std::is_same<QT, BF16>::value;
    static constexpr int NE = G == 1 ? 1 : 2;                     // heads a lane works on
    static_assert(UB == 1 || UB == 2 || UB == 4, "whole blocks per unit");
    static_assert(G == 1 || G == 2 || G == 4 || G == 8, "heads fill at most 8 MMA columns");
    static_assert(MIN_CTAS * (SMEM + 1024) <= 233472, "the CTAs of an SM share 228 KB");
    static_assert(SMEM_ONE + 1024 <= 233472 && G * D * 4 <= STAGE, "a CTA per segment");
    static_assert((kOneWarps + 2) * G * 8 <= kPrefixBytes && NS >= 2, "(m, l) take the prefix's place");
};

struct Params {
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const float* k_scales;
    const float* v_scales;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* lists;        // kList: [batch, hkv, max_list] block indices of the sequence
    const int32_t* list_lens;    // kList: [batch]
    void* out;
    const float* mass_in;        // kMass: [batch, hkv, mb * 16] or nullptr (zeros)
    float* mass_out;             // kMass
    float* scores;               // kMass: [batch, hkv, mb * 16, G], log2 units
    float* part_o;               // [slots, G, D], slot = segment + worker
    float* part_ml;              // [slots, G, 2]
    int32_t* ws_prefix;          // [batch + 1] unit prefix, for the join
    uint32_t* status;
    int batch, hq, hkv, mb, num_blocks, max_list, workers;
    float qscale;                // softmax_scale * log2(e)
    uint64_t wait_ns;            // limit of each bounded wait on a stage (kWaitLimitNs)
    int stall_worker;            // test hook: this worker's first stage expects 16 bytes that
                                 // no copy delivers, so its wait runs out (-1: none)
    int keep_scores;             // kMass: the scores fit L2
    int lslices;                 // 2^lslices merging CTAs share a segment's output
    int cluster;                 // ONE: CTAs per segment
    int mass_ctas;               // join: CTAs that turn scores into weights (kMass)
    int segs_per_cta, seg_ctas;  // join: segments per merging CTA, merging CTAs
};

__host__ __device__ inline int prefix_stride(int batch) {
    return batch <= kPrefixEntries ? 1 : (batch + kPrefixEntries - 1) / kPrefixEntries;
}
__host__ __device__ inline int prefix_chunks(int batch) {
    const int st = prefix_stride(batch);
    return (batch + st - 1) / st;
}

// Workers that get units: at most one per kMinUnits units, so that every range
// is non-empty and short calls are not cut into single-block pieces.
constexpr long long kMinUnits = 4;
__host__ __device__ inline long long eff_workers(long long U, long long W) {
    const long long cap = U / kMinUnits;
    return cap < 1 ? 1 : (cap < W ? cap : W);
}
// Worker whose range holds unit u: the largest w with floor(w U / W) <= u.
__device__ __forceinline__ long long worker_of(long long u, long long U, long long W) {
    return ((u + 1) * W - 1) / U;
}

__device__ __forceinline__ int clamp_to(int n, int most, uint32_t* status, bool flag) {
    if (n < 0 || n > most) {
        if (flag) flag_status(status, PKV_DEV_BAD_LENGTH);
        n = n < 0 ? 0 : most;
    }
    return n;
}
__device__ __forceinline__ int seq_len(const Params& p, int b, bool flag) {
    return clamp_to(__ldg(p.context_lens + b), p.mb * kBlockSize, p.status, flag);
}
// Entries (16-token blocks) of sequence b.
template <int M>
__device__ __forceinline__ int seq_entries(const Params& p, int b, bool flag) {
    if constexpr (M == kList) return clamp_to(__ldcg(p.list_lens + b), p.max_list, p.status, flag);
    else return (seq_len(p, b, flag) + kBlockSize - 1) / kBlockSize;
}
template <int M, int UB>
__device__ __forceinline__ int seq_units(const Params& p, int b, bool flag) {
    return (seq_entries<M>(p, b, flag) + UB - 1) / UB;
}

// Exclusive prefix of the sequences' units. Shared memory keeps
// prefix[c] = P[c * stride] and prefix[chunks] = P[batch]; CTA 0 writes all of
// P to ws_prefix for the join, and flags lengths that do not fit.
template <int M, int UB, int THREADS>
__device__ void build_prefix(const Params& p, int* warp_tot, int* prefix) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int chunk = (p.batch + THREADS - 1) / THREADS;
    const int lo = min(p.batch, t * chunk), hi = min(p.batch, lo + chunk);
    const bool zero = blockIdx.x == 0;
    int sum = 0;
    for (int i = lo; i < hi; ++i) {
        sum += seq_units<M, UB>(p, i, zero);
        if (M == kList && zero) seq_len(p, i, true);
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFull, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) warp_tot[warp] = inc;
    __syncthreads();
    int run = inc - sum;
    for (int w = 0; w < warp; ++w) run += warp_tot[w];
    const int stride = prefix_stride(p.batch);
    for (int i = lo; i < hi; ++i) {
        if (i % stride == 0) prefix[i / stride] = run;
        if (zero) p.ws_prefix[i] = run;
        run += seq_units<M, UB>(p, i, false);
    }
    if (t == THREADS - 1) {
        prefix[prefix_chunks(p.batch)] = run;
        if (zero) p.ws_prefix[p.batch] = run;
    }
    __syncthreads();
}

// Unit u -> sequence b, kv head, unit j of the segment's nu units. b is the
// last sequence whose first unit is <= u; it has units, since u < U.
template <int M, int UB>
__device__ __forceinline__ void find_unit(long long u, const int* prefix, const Params& p, int& b,
                                          int& kvh, int& j, int& nu) {
    const int x = int(u / p.hkv);
    const int stride = prefix_stride(p.batch), chunks = prefix_chunks(p.batch);
    int lo = 0;
    static_assert(kPrefixEntries <= 256, "search width");
    for (int step = 1 << 7; step; step >>= 1)
        if (lo + step < chunks && prefix[lo + step] <= x) lo += step;
    int first = prefix[lo];
    if (stride == 1) {
        b = lo;
        nu = prefix[lo + 1] - first;
    } else {
        b = lo * stride;
        const int last = min(b + stride, p.batch) - 1;
        nu = seq_units<M, UB>(p, b, false);
        while (b < last && x >= first + nu) {
            first += nu;
            nu = seq_units<M, UB>(p, ++b, false);
        }
    }
    const int r = int(u - (long long)p.hkv * first);
    kvh = r / nu;
    j = r - kvh * nu;
}

template <typename QT, int N>
__device__ __forceinline__ void store_row(void* out, long long off, const float2* v, float s) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = pack2<QT>(v[i].x * s, v[i].y * s);
    uint16_t* dst = static_cast<uint16_t*>(out) + off;
    if constexpr (N % 8 == 0) {
#pragma unroll
        for (int i = 0; i < N / 8; ++i)
            reinterpret_cast<uint4*>(dst)[i] =
                make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
        static_assert(N == 4, "row pieces of 4 or a multiple of 8 values");
        *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    }
}

// Two INT8 codes as fp16, exact: the byte c + 128 under 0x64 is 1152 + c, and
// 1152 comes off again. (Leaving the bias in the products and taking it off
// the sums is cheaper, but the sums then round at 1152 times the size of what
// is wanted: 2e-5 of a weight, against 1e-6 this way.)
__device__ __forceinline__ uint32_t codes_h2(uint32_t biased, uint32_t sel) {
    const uint32_t w = i8x2_biased_h2(biased, sel);
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&w), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint4 sel4(bool c, const uint4& a, const uint4& b) {
    return make_uint4(c ? a.x : b.x, c ? a.y : b.y, c ? a.z : b.z, c ? a.w : b.w);
}

// bulk_g2s with an L2 cache policy.
__device__ __forceinline__ void bulk_g2s_hint(uint32_t dst, const void* src, uint32_t bytes,
                                              uint32_t bar, uint64_t policy) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
                 " [%0], [%1], %2, [%3], %4;"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar), "l"(policy) : "memory");
}

// A sum l of 0 holds nothing; one that is NaN (a NaN or infinite score, whose
// maximum may be -inf) stays NaN through every merge, so the row shows it.
__device__ __forceinline__ float reciprocal(float l) { return l == 0.f ? 0.f : 1.f / l; }

__device__ __forceinline__ void merge_ml(float& m, float& l, float m2, float l2) {
    if (l2 == 0.f) return;
    const float mn = fmaxf(m, m2);
    l = l * fast_exp2(m - mn) + l2 * fast_exp2(m2 - mn);
    m = mn;
}

// kMass: weights of tokens i = t, t + n, ... of [t0, t1) of segment seg, whose
// head h has its maximum in ml[h].x and 1 / l in ml[h].y.
template <int G>
__device__ __forceinline__ void weigh(const Params& p, long long seg, int t0, int t1, int t, int n,
                                      const float2 (&ml)[G]) {
    const long long row = seg * p.mb * kBlockSize;
    const float* sc = p.scores + row * G;
    float* out = p.mass_out + row;
    const float* in = p.mass_in ? p.mass_in + row : nullptr;
    // tokens in flight per thread: all loads before the stores, since mass_in
    // may be mass_out
    constexpr int R = G == 8 ? 2 : 4;
    for (int i0 = t0 + t; i0 < t1; i0 += R * n) {
        float x[R][G], old[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = i0 + r * n;
            old[r] = 0.f;
#pragma unroll
            for (int h = 0; h < G; ++h) x[r][h] = -INFINITY;
            if (i >= t1) continue;
            if (in) old[r] = in[i];
            if constexpr (G >= 4) {
#pragma unroll
                for (int c = 0; c < G / 4; ++c) {
                    const float4 v = reinterpret_cast<const float4*>(sc)[(long long)i * (G / 4) + c];
                    x[r][4 * c] = v.x; x[r][4 * c + 1] = v.y; x[r][4 * c + 2] = v.z; x[r][4 * c + 3] = v.w;
                }
            } else if constexpr (G == 2) {
                const float2 v = reinterpret_cast<const float2*>(sc)[i];
                x[r][0] = v.x; x[r][1] = v.y;
            } else {
                x[r][0] = sc[i];
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = i0 + r * n;
            if (i >= t1) continue;
            float add = 0.f;
#pragma unroll
            for (int h = 0; h < G; ++h) add += fast_exp2(x[r][h] - ml[h].x) * ml[h].y;
            out[i] = old[r] + add;
        }
    }
}

// ------------------------------------------------------------ cluster ---
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A shared-memory address of this CTA as the same place of CTA `rank`'s.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float2 load_remote2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 load_remote4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// Fold the state (m2, l2, o2) into (m, l, o); l2 = 0 holds nothing.
__device__ __forceinline__ void fold(float& m, float& l, float4& o, float m2, float l2, const float4& o2) {
    if (l2 == 0.f) return;
    const float mn = fmaxf(m, m2), a = fast_exp2(m - mn), c = fast_exp2(m2 - mn);
    l = l * a + l2 * c;
    o.x = o.x * a + o2.x * c; o.y = o.y * a + o2.y * c;
    o.z = o.z * a + o2.z * c; o.w = o.w * a + o2.w * c;
    m = mn;
}

// ONE: the end of the cluster that has segment (sequence b, kv head kvh) to
// itself. Warp w left (m, l) of its share in s_ml[w][G] (l = 0: none) and o in
// the first stage of its region, `stride` bytes from the next warp's. The CTA
// folds its warps' states into its second stage and s_ml[kOneWarps][G]; the
// cluster's CTAs then share the output, and each weighs the tokens [t0, t1) whose
// scores it wrote.
template <typename QT, int D, int G, int M>
__device__ __forceinline__ void one_out(const Params& p, int b, int kvh, int rank, float2* s_ml,
                                        unsigned char* regions, int stride, int stage, int t0, int t1) {
    constexpr int Q = D / 4, ITEMS = G * Q;
    static_assert(ITEMS <= 32 * kOneWarps, "a thread per float4 of the output");
    const int t = threadIdx.x, h = t / Q;
    float2* s_cta = s_ml + kOneWarps * G;
    float4* o_cta = reinterpret_cast<float4*>(regions + stage);
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t < ITEMS) {
#pragma unroll
        for (int w = 0; w < kOneWarps; ++w) {
            const float2 ml = s_ml[w * G + h];
            if (ml.y == 0.f) continue;             // nothing was left there
            fold(m, l, o, ml.x, ml.y, reinterpret_cast<const float4*>(regions + w * stride)[t]);
        }
    }
    const int n = p.cluster;
    if (n > 1) {
        if (t < ITEMS) {
            o_cta[t] = o;
            if (t % Q == 0) s_cta[h] = make_float2(m, l);
        }
        cluster_sync();
        m = -INFINITY;
        l = 0.f;
        o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t < ITEMS && t % n == rank) {
            for (int r = 0; r < n; ++r) {
                const float2 ml = load_remote2(map_rank(smem_addr(s_cta + h), r));
                fold(m, l, o, ml.x, ml.y, load_remote4(map_rank(smem_addr(o_cta + t), r)));
            }
        }
    }
    if (t < ITEMS && t % n == rank) {
        const float2 v[2] = {make_float2(o.x, o.y), make_float2(o.z, o.w)};
        store_row<QT, 4>(p.out, ((long long)b * p.hq + kvh * G) * D + t * 4, v, reciprocal(l));
    }
    if constexpr (M == kMass) {
        float2* s_fin = s_cta + G;
        if (t < G) {
            m = -INFINITY;
            l = 0.f;
            for (int r = 0; r < (n > 1 ? n : kOneWarps); ++r) {
                const float2 ml = n > 1 ? load_remote2(map_rank(smem_addr(s_cta + t), r)) : s_ml[r * G + t];
                merge_ml(m, l, ml.x, ml.y);
            }
            s_fin[t] = make_float2(m == -INFINITY ? 0.f : m, reciprocal(l));
        }
        __syncthreads();
        float2 ml[G];
#pragma unroll
        for (int k = 0; k < G; ++k) ml[k] = s_fin[k];
        weigh<G>(p, (long long)b * p.hkv + kvh, t0, t1, t, 32 * kOneWarps, ml);
    }
    if (n > 1) cluster_sync();     // nobody leaves while its memory is read
}

// ONE: a cluster of p.cluster CTAs has one segment to itself, shared by their
// kOneWarps warps each, and finishes it: no prefix, no workspace for pieces and no
// join. For calls of few and short segments, which are all latency.
template <typename KV, typename QT, int D, int G, int M, bool ONE>
__global__ void __launch_bounds__(ONE ? 32 * kOneWarps : Cfg<KV, QT, D, G>::THREADS,
                                  ONE ? 1 : Cfg<KV, QT, D, G>::MIN_CTAS)
ctx_split_kernel(const Params p) {
    using C = Cfg<KV, QT, D, G>;
    using MT = typename std::conditional<C::kI8, F16, KV>::type;   // mma operand type
    constexpr int UB = C::UB;
    extern __shared__ __align__(128) unsigned char smem[];
    int* warp_tot = reinterpret_cast<int*>(smem);
    int* prefix = warp_tot + kMaxWarps;
    float2* s_ml = reinterpret_cast<float2*>(smem);   // ONE: [kOneWarps][G]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * (ONE ? kOneWarps : C::WARPS) + warp;
    const int one_seg = ONE ? int(blockIdx.x) / p.cluster : 0, rank = ONE ? int(blockIdx.x) - one_seg * p.cluster : 0;
    const int one_b = one_seg / p.hkv, one_kvh = one_seg - one_b * p.hkv;
    long long u0, u1;
    int one_nu = 0;
    griddep_wait();
    if constexpr (ONE) {
        const bool flag = one_kvh == 0 && rank == 0 && threadIdx.x == 0;
        one_nu = seq_units<M, UB>(p, one_b, flag);
        if (M == kList && flag) seq_len(p, one_b, true);
        const int share = rank * kOneWarps + warp, shares = p.cluster * kOneWarps;
        u0 = (long long)share * one_nu / shares;
        u1 = (long long)(share + 1) * one_nu / shares;
        if (lane < G) s_ml[warp * G + lane] = make_float2(-INFINITY, 0.f);
    } else {
        griddep_launch_dependents();
        build_prefix<M, UB, C::THREADS>(p, warp_tot, prefix);
        const long long U = (long long)prefix[prefix_chunks(p.batch)] * p.hkv;
        const long long W = eff_workers(U, p.workers);
        if (w >= W || U == 0) return;
        u0 = w * U / W;
        u1 = (w + 1) * U / W;
    }

    unsigned char* region = smem + kPrefixBytes + warp * C::WARP_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(region + C::OFF_BAR);
    int4* meta = reinterpret_cast<int4*>(region + C::OFF_META);
    float2* scl = reinterpret_cast<float2*>(region + C::OFF_SCL);
    float* pbuf = reinterpret_cast<float*>(region + C::OFF_P);
    if (lane == 0) {
#pragma unroll
        for (int s = 0; s < C::NS; ++s) mbar_init(smem_addr(&bars[s]), C::ARRIVALS);
        fence_mbar_init();
    }
    __syncwarp();

    // kMass: where the scores fit L2, K and V, which pass through it once, are
    // evicted first, so that the join finds the scores there (33 MB of them: 126.1
    // instead of 126.7 us, and 120.9 instead of 125.8 where calls repeat the same
    // inputs; 134 MB: 383 instead of 380).
    uint64_t policy = 0;
    if constexpr (M == kMass) {
        if (p.keep_scores) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
        else asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
    }

    // ---- producer. Lane i holds unit base + i: physical blocks (-1: none) and
    // their valid tokens, 32 units ahead of the copies.
    struct Ahead {
        int b, kvh, j, blk[UB], nv;   // nv: tokens of block i << 6 i, last unit << 24
    };
    auto fetch = [&](long long base) {
        Ahead a;
        const long long u = base + lane;
        a.b = a.kvh = a.j = a.nv = 0;
#pragma unroll
        for (int i = 0; i < UB; ++i) a.blk[i] = -1;
        if (u < u1) {
            int nu;
            if constexpr (ONE) {
                a.b = one_b;
                a.kvh = one_kvh;
                a.j = int(u);
                nu = one_nu;
            } else {
                find_unit<M, UB>(u, prefix, p, a.b, a.kvh, a.j, nu);
            }
            const int L = seq_len(p, a.b, false), nblk = (L + kBlockSize - 1) / kBlockSize;
            const int entries = (M == kList) ? seq_entries<M>(p, a.b, false) : nblk;
            if (a.j == nu - 1) a.nv = 1 << 24;
#pragma unroll
            for (int i = 0; i < UB; ++i) {
                const int e = UB * a.j + i;
                if (e >= entries) continue;
                int id = e;
                if constexpr (M == kList)
                    id = __ldcg(p.lists + ((long long)a.b * p.hkv + a.kvh) * p.max_list + e);
                if (unsigned(id) >= unsigned(nblk)) {     // kList only: not a block of the sequence
                    flag_status(p.status, PKV_DEV_BAD_INDEX);
                    continue;
                }
                const int blk = __ldg(p.block_tables + (long long)a.b * p.mb + id);
                if (unsigned(blk) >= unsigned(p.num_blocks)) {
                    flag_status(p.status, PKV_DEV_BAD_BLOCK);
                    continue;
                }
                a.blk[i] = blk;
                a.nv |= min(kBlockSize, L - id * kBlockSize) << (6 * i);
            }
        }
        return a;
    };
    long long cbase = u0;
    Ahead cur = fetch(cbase), nxt = fetch(cbase + 32);

    auto issue = [&](long long u, int s, uint32_t extra_tx) {
        int idx = int(u - cbase);
        if (idx >= 32) {
            cbase += 32;
            cur = nxt;
            nxt = fetch(cbase + 32);
            idx -= 32;
        }
        const int b = __shfl_sync(kFull, cur.b, idx), kvh = __shfl_sync(kFull, cur.kvh, idx);
        const int j = __shfl_sync(kFull, cur.j, idx), nv = __shfl_sync(kFull, cur.nv, idx);
        // lane c copies K (c < UB) or V of block c % UB
        int blk = -1;
#pragma unroll
        for (int i = 0; i < UB; ++i) {
            const int x = __shfl_sync(kFull, cur.blk[i], idx);
            if (lane % UB == i) blk = x;
        }
        const uint32_t bar = smem_addr(&bars[s]);
        const bool first = (u == u0) || (j == 0);   // first unit of a piece
        if (lane == 0) {
            int n = 0;
#pragma unroll
            for (int i = 0; i < UB; ++i) n += ((nv >> (6 * i)) & 63) != 0;
            meta[s] = make_int4(b, kvh | (first ? 1 << 17 : 0), j, nv);
            const uint32_t tx = n * 2 * C::TILE + extra_tx;
            if (tx) mbar_arrive_expect_tx(bar, tx);
            else mbar_arrive(bar);
        }
        __syncwarp();
        if (lane < 2 * UB) {
            const long long tile = (long long)blk * p.hkv + kvh;
            if (blk >= 0) {
                const void* src = lane < UB ? p.k_cache : p.v_cache;
                const uint32_t dst = smem_addr(region + s * C::STAGE) + lane * C::TILE;
                const char* from = static_cast<const char*>(src) + tile * C::TILE;
                if constexpr (M == kMass) bulk_g2s_hint(dst, from, C::TILE, bar, policy);
                else bulk_g2s(dst, from, C::TILE, bar);
                if constexpr (C::kI8)
                    cp_async_4(smem_addr(scl + UB * s + lane % UB) + 4 * (lane / UB),
                               (lane < UB ? p.k_scales : p.v_scales) + tile);
            }
            if constexpr (C::kI8) cp_async_arrive_noinc(bar);
        }
        if (first && lane < G * D / 32)   // the piece's q rows, 64 bytes a lane, into L2
            asm volatile("prefetch.global.L2 [%0];" ::"l"(
                static_cast<const uint16_t*>(p.q) + ((long long)b * p.hq + kvh * G) * D + 32 * lane));
    };

    // ---- consumer. Lane (gq, tq) = (lane / 4, lane % 4) holds the scores of
    // tokens gq, gq + 8 and heads 2tq, 2tq + 1, and accumulates dims
    // [gq D/8, (gq+1) D/8) of O for those two heads.
    constexpr int NT = D / 16;                   // m-tiles of P V, and k-steps of the scores
    constexpr int DL = D / 8;
    const int gq = lane >> 2, tq = lane & 3;
    uint32_t qb[NT][2];
    float qs[2] = {p.qscale, p.qscale};   // score factor of heads 2tq, 2tq + 1
    float m[2] = {-INFINITY, -INFINITY}, lsum[2] = {0.f, 0.f};
    float oa[NT][4];
    int pb = -1, pkvh = 0, first_j = 0;
    bool last_seen = false;
    // INT8: P carries the block's V scale into fp16, so O is kept in units of
    // 2^vexp, chosen from the piece's first scales so that a weight of 1 sits
    // near 2^13 (small weights stay in fp16's normal range; less for scales below
    // 2^-113, since 2^-vexp is at most 2^126) and raised when a later scale would
    // pass 2^14. vmul = 2^-vexp, 0 until chosen.
    int vexp = 0;
    float vmul = 0.f;

    auto finalize = [&]() {
        const long long seg = (long long)pb * p.hkv + pkvh;
        const bool whole = first_j == 0 && last_seen;
        float lh[2] = {lsum[0], lsum[1]};   // [1] is unused with one head
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
#pragma unroll
            for (int e = 0; e < C::NE; ++e) lh[e] += __shfl_xor_sync(kFull, lh[e], off);
        const float up = C::kI8 ? ldexpf(1.f, vexp) : 1.f;
#pragma unroll
        for (int e = 0; e < C::NE; ++e) {
            const int h = 2 * tq + e;
            if (h >= G) continue;
            const long long slot = seg + w;
            if constexpr (ONE) {          // the warp's first stage is free by now
                float4* dst = reinterpret_cast<float4*>(region) + (h * D + gq * DL) / 4;
#pragma unroll
                for (int i = 0; i < NT / 2; ++i)
                    dst[i] = make_float4(oa[2 * i][e] * up, oa[2 * i][2 + e] * up,
                                         oa[2 * i + 1][e] * up, oa[2 * i + 1][2 + e] * up);
                if (gq == 0) s_ml[warp * G + h] = make_float2(m[e], lh[e]);
                continue;
            }
            if (whole) {
                const float inv = reciprocal(lh[e]);     // up / l could be denormal
                float2 v[NT];
#pragma unroll
                for (int i = 0; i < NT; ++i) v[i] = make_float2(oa[i][e] * inv, oa[i][2 + e] * inv);
                store_row<QT, DL>(p.out, ((long long)pb * p.hq + pkvh * G + h) * D + gq * DL, v, up);
            } else {
                float4* dst = reinterpret_cast<float4*>(p.part_o + (slot * G + h) * D + gq * DL);
#pragma unroll
                for (int i = 0; i < NT / 2; ++i)
                    dst[i] = make_float4(oa[2 * i][e] * up, oa[2 * i][2 + e] * up,
                                         oa[2 * i + 1][e] * up, oa[2 * i + 1][2 + e] * up);
            }
            // kMass: the join needs every segment's (M, l)
            if ((M == kMass || !whole) && gq == 0)
                *reinterpret_cast<float2*>(p.part_ml + (slot * G + h) * 2) = make_float2(m[e], lh[e]);
        }
    };

    for (int s = 0; s < C::NS; ++s)
        if (u0 + s < u1) issue(u0 + s, s, (s == 0 && w == p.stall_worker) ? 16u : 0u);
    long long u_issue = (u0 + C::NS < u1) ? u0 + C::NS : u1;
    uint32_t parity = 0;
    bool aborted = false;
    long long u = u0;
    int s = 0;
    for (; u < u1; ++u, s = (s + 1 == C::NS) ? 0 : s + 1) {
        const bool got = mbar_wait_bounded(smem_addr(&bars[s]), (parity >> s) & 1u, p.wait_ns);
        if (!__all_sync(kFull, got)) {
            if (lane == 0) flag_status(p.status, PKV_DEV_TIMEOUT);
            aborted = true;
            break;
        }
        parity ^= 1u << s;
        const int4 mt = meta[s];
        if (mt.y >> 17) {   // first unit of a new piece
            if (pb >= 0) finalize();
            pb = mt.x;
            pkvh = mt.y & 0xffff;
            first_j = mt.z;
            const uint16_t* qs16 = static_cast<const uint16_t*>(p.q) + ((long long)pb * p.hq + pkvh * G) * D;
            // q^T as the B operand, the contraction index permuted so that one
            // 16-byte load of a K row serves several k-steps. 16-bit: k-steps 2c,
            // 2c + 1 of lane tq read dims 32c + 8tq + [0, 4) and + [4, 8). INT8:
            // k-step kk of lane tq reads dims 16tq + 4(kk%4) + 64(kk/4) + [0, 4).
            // INT8 codes meet q in fp16; a bf16 head is brought into its range by a
            // power of two, which its score factor qs takes back.
            float amax = 0.f;
#pragma unroll
            for (int kk = 0; kk < NT; ++kk) {
                qb[kk][0] = qb[kk][1] = 0u;
                const int d0 = C::kI8 ? 16 * tq + 4 * (kk % 4) + 64 * (kk / 4)
                                      : 32 * (kk / 2) + 8 * tq + 4 * (kk % 2);
                if (gq < G) {
                    const uint2 x = __ldg(reinterpret_cast<const uint2*>(qs16 + gq * D + d0));
                    qb[kk][0] = x.x;
                    qb[kk][1] = x.y;
                }
                if constexpr (C::kFit) {
                    const float2 f0 = unpack2(QT{}, qb[kk][0]), f1 = unpack2(QT{}, qb[kk][1]);
                    amax = fmaxf(fmaxf(fmaxf(amax, fabsf(f0.x)), fmaxf(fabsf(f0.y), fabsf(f1.x))), fabsf(f1.y));
                }
            }
            if constexpr (C::kFit) {           // a head's dims lie in lanes 4 gq + [0, 4)
                amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
                const float2 fit = fit_half(amax);
#pragma unroll
                for (int kk = 0; kk < NT; ++kk)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 f = unpack2(QT{}, qb[kk][i]);
                        qb[kk][i] = pack2<F16>(f.x * fit.x, f.y * fit.x);
                    }
#pragma unroll
                for (int e = 0; e < C::NE; ++e)
                    qs[e] = p.qscale * __shfl_sync(kFull, fit.y, (8 * tq + 4 * e) & 31);
            }
#pragma unroll
            for (int e = 0; e < C::NE; ++e) { m[e] = -INFINITY; lsum[e] = 0.f; }
#pragma unroll
            for (int i = 0; i < NT; ++i) oa[i][0] = oa[i][1] = oa[i][2] = oa[i][3] = 0.f;
            vexp = 0;
            vmul = 0.f;
        }
        last_seen = (mt.w >> 24) & 1;

        const unsigned char* kt = region + s * C::STAGE;
        const unsigned char* vt = kt + UB * C::TILE;
        int nv[UB];
#pragma unroll
        for (int i = 0; i < UB; ++i) nv[i] = (mt.w >> (6 * i)) & 63;
        // kMass keeps the scores of skipped blocks too (-inf: weight 0)
        if (M == kMass || (mt.w & 0xffffff)) {
            // ---- scores, two accumulator chains (even / odd k-steps). A row is
            // a multiple of 128 bytes, so all rows share the bank mapping: lanes
            // of odd gq read the two halves of a 128-byte span in the other
            // order, which spreads a quarter warp over all banks.
            float acc[UB][2][4];
#pragma unroll
            for (int i = 0; i < UB; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c) acc[i][c][0] = acc[i][c][1] = acc[i][c][2] = acc[i][c][3] = 0.f;
            float ksc[UB], vsc[UB];
            if constexpr (!C::kI8) {
                const bool kswap = (gq & 1) != 0;
#pragma unroll
                for (int bi = 0; bi < UB; ++bi) {
                    ksc[bi] = vsc[bi] = 1.f;
                    const unsigned char* kb = kt + bi * C::TILE;
#pragma unroll
                    for (int c2 = 0; c2 < D / 32; c2 += 2) {
                        uint4 y[2][2];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int off = 64 * (c2 + (h ^ (kswap ? 1 : 0))) + 16 * tq;
                            y[h][0] = *reinterpret_cast<const uint4*>(kb + gq * C::ROW + off);
                            y[h][1] = *reinterpret_cast<const uint4*>(kb + (gq + 8) * C::ROW + off);
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int c = c2 + h;
                            const uint4 x0 = sel4(kswap, y[h ^ 1][0], y[h][0]);
                            const uint4 x1 = sel4(kswap, y[h ^ 1][1], y[h][1]);
                            const uint32_t a0[4] = {x0.x, x1.x, x0.y, x1.y};
                            const uint32_t a1[4] = {x0.z, x1.z, x0.w, x1.w};
                            mma16816<MT>(acc[bi][0], a0, qb[2 * c][0], qb[2 * c][1]);
                            mma16816<MT>(acc[bi][1], a1, qb[2 * c + 1][0], qb[2 * c + 1][1]);
                        }
                    }
                }
            } else {
                float vmax = 0.f;
#pragma unroll
                for (int i = 0; i < UB; ++i) {
                    const float2 sc = scl[UB * s + i];
                    ksc[i] = nv[i] ? sc.x : 0.f;
                    vsc[i] = nv[i] ? sc.y : 0.f;
                    vmax = fmaxf(vmax, vsc[i]);
                }
                if (vmax > 0.f && (vmul == 0.f || vmax * vmul >= 16384.f)) {   // warp-uniform
                    int ex;
                    frexpf(vmax, &ex);          // vmax < 2^ex
                    const int nexp = max(ex - 13, -126);   // 2^-nexp is finite
                    if (vmul != 0.f) {
                        const float r = ldexpf(1.f, vexp - nexp);
#pragma unroll
                        for (int i = 0; i < NT; ++i) {
                            oa[i][0] *= r; oa[i][1] *= r; oa[i][2] *= r; oa[i][3] *= r;
                        }
                    }
                    vexp = nexp;
                    vmul = ldexpf(1.f, -nexp);
                }
#pragma unroll
                for (int i = 0; i < UB; ++i) vsc[i] *= vmul;
#pragma unroll
                for (int bi = 0; bi < UB; ++bi) {
                    const unsigned char* kb = kt + bi * C::TILE;
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        const uint4 y0 = *reinterpret_cast<const uint4*>(kb + gq * C::ROW + 64 * c + 16 * tq);
                        const uint4 y1 = *reinterpret_cast<const uint4*>(kb + (gq + 8) * C::ROW + 64 * c + 16 * tq);
                        const uint32_t w0[4] = {y0.x, y0.y, y0.z, y0.w}, w1[4] = {y1.x, y1.y, y1.z, y1.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int kk = 4 * c + k;
                            const uint32_t x0 = w0[k] ^ 0x80808080u, x1 = w1[k] ^ 0x80808080u;
                            const uint32_t a[4] = {codes_h2(x0, 0x4140), codes_h2(x1, 0x4140),
                                                   codes_h2(x0, 0x4342), codes_h2(x1, 0x4342)};
                            mma16816<MT>(acc[bi][kk & 1], a, qb[kk][0], qb[kk][1]);
                        }
                    }
                }
            }
            // ---- V rows of the lane, read before the softmax's shared stores
            constexpr int VW = C::kI8 ? DL / 4 : DL / 2;    // words per row
            const int vswap = (!C::kI8 && DL / 8 == 2) ? (tq & 1) : 0;
            uint32_t vw[UB][4][VW];
#pragma unroll
            for (int bi = 0; bi < UB; ++bi)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = 2 * tq + (i & 1) + 8 * (i >> 1);
                    const unsigned char* row = vt + bi * C::TILE + t * C::ROW + gq * (C::ROW / 8);
                    if constexpr (VW == 2) {
                        const uint2 x = *reinterpret_cast<const uint2*>(row);
                        vw[bi][i][0] = x.x; vw[bi][i][1] = x.y;
                    } else {
#pragma unroll
                        for (int c = 0; c < VW / 4; ++c) {
                            const uint4 x = *reinterpret_cast<const uint4*>(row + 16 * (c ^ vswap));
                            vw[bi][i][4 * c] = x.x; vw[bi][i][4 * c + 1] = x.y;
                            vw[bi][i][4 * c + 2] = x.z; vw[bi][i][4 * c + 3] = x.w;
                        }
                    }
                }
            // ---- masked scores in log2 units
            float sv[UB][2][2];   // [block][token gq / gq + 8][head 2tq + e]
#pragma unroll
            for (int bi = 0; bi < UB; ++bi) {
#pragma unroll
                for (int e = 0; e < C::NE; ++e) {
                    const float sk = (C::kFit ? qs[e] : p.qscale) * ksc[bi];
                    const bool hv = 2 * tq + e < G;
                    const float s0 = acc[bi][0][e] + acc[bi][1][e];
                    const float s1 = acc[bi][0][2 + e] + acc[bi][1][2 + e];
                    sv[bi][0][e] = (hv && gq < nv[bi]) ? s0 * sk : -INFINITY;
                    sv[bi][1][e] = (hv && gq + 8 < nv[bi]) ? s1 * sk : -INFINITY;
                }
                if constexpr (M == kMass) {
                    const int entry = UB * mt.z + bi;
                    if (UB == 1 || entry < p.mb) {   // a two-block unit may end past the table
                        const long long row = ((long long)pb * p.hkv + pkvh) * p.mb + entry;
                        float* dst = p.scores + row * kBlockSize * G + 2 * tq;
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            if constexpr (G == 1) {
                                if (tq == 0) dst[gq + 8 * r] = sv[bi][r][0];
                            } else if (2 * tq < G) {
                                *reinterpret_cast<float2*>(dst + (gq + 8 * r) * G) =
                                    make_float2(sv[bi][r][0], sv[bi][r][1]);
                            }
                        }
                    }
                }
            }
            // ---- running maximum and sum; P into shared memory
            float alpha[2];
#pragma unroll
            for (int e = 0; e < C::NE; ++e) {
                float mx = fmaxf(sv[0][0][e], sv[0][1][e]);
#pragma unroll
                for (int bi = 1; bi < UB; ++bi) mx = fmaxf(mx, fmaxf(sv[bi][0][e], sv[bi][1][e]));
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, off));
                const float mn = fmaxf(m[e], mx);
                const float base = mn == -INFINITY ? 0.f : mn;   // nothing valid yet: all 2^-inf
                alpha[e] = mn == -INFINITY ? 1.f : fast_exp2(m[e] - mn);
                m[e] = mn;
                float ls = lsum[e] * alpha[e];
#pragma unroll
                for (int bi = 0; bi < UB; ++bi) {
                    const float p0 = fast_exp2(sv[bi][0][e] - base), p1 = fast_exp2(sv[bi][1][e] - base);
                    ls = ls + p0 + p1;
                    if (2 * tq + e < G) {
                        float* dst = pbuf + (2 * tq + e) * C::PS + kBlockSize * bi;
                        dst[gq] = C::kI8 ? p0 * vsc[bi] : p0;
                        dst[gq + 8] = C::kI8 ? p1 * vsc[bi] : p1;
                    }
                }
                lsum[e] = ls;
            }
            if constexpr (C::NE == 1) alpha[1] = 1.f;
            if (__any_sync(kFull, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    oa[i][0] *= alpha[0]; oa[i][1] *= alpha[1];
                    oa[i][2] *= alpha[0]; oa[i][3] *= alpha[1];
                }
            }
            __syncwarp();
            // ---- O^T += V^T P^T: A rows gq, gq + 8 of m-tile i are dims
            // gq DL + 2i, + 1; columns are tokens 2tq, 2tq + 1 | + 8.
#pragma unroll
            for (int bi = 0; bi < UB; ++bi) {
                uint32_t ph[2] = {0u, 0u}, pl[2] = {0u, 0u};
                if (gq < G) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float2 f = *reinterpret_cast<const float2*>(
                            pbuf + gq * C::PS + kBlockSize * bi + 2 * tq + 8 * k);
                        ph[k] = pack2<MT>(f.x, f.y);
                        if constexpr (C::kTwoParts) {
                            const float2 r = unpack2(MT{}, ph[k]);
                            pl[k] = pack2<MT>(f.x - r.x, f.y - r.y);
                        }
                    }
                }
                if constexpr (!C::kI8) {
                    // rows past the context may hold anything, and 0 * NaN
                    // would poison the sum: they become zeros
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool keep = 2 * tq + (i & 1) + 8 * (i >> 1) < nv[bi];
#pragma unroll
                        for (int c = 0; c < VW; ++c) {
                            if (!keep) vw[bi][i][c] = 0u;
                        }
                        if constexpr (DL / 8 == 2) {
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const uint32_t x = vw[bi][i][c], y = vw[bi][i][4 + c];
                                vw[bi][i][c] = vswap ? y : x;
                                vw[bi][i][4 + c] = vswap ? x : y;
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const uint32_t a[4] = {__byte_perm(vw[bi][0][i], vw[bi][1][i], 0x5410),
                                               __byte_perm(vw[bi][0][i], vw[bi][1][i], 0x7632),
                                               __byte_perm(vw[bi][2][i], vw[bi][3][i], 0x5410),
                                               __byte_perm(vw[bi][2][i], vw[bi][3][i], 0x7632)};
                        mma16816<MT>(oa[i], a, ph[0], ph[1]);
                        mma16816<MT>(oa[i], a, pl[0], pl[1]);
                    }
                } else {
                    // any byte is a finite code and a masked token's P is 0
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
                        const uint32_t x = __byte_perm(vw[bi][0][i / 2], vw[bi][1][i / 2], sel) ^ 0x80808080u;
                        const uint32_t y = __byte_perm(vw[bi][2][i / 2], vw[bi][3][i / 2], sel) ^ 0x80808080u;
                        const uint32_t a[4] = {codes_h2(x, 0x4140), codes_h2(x, 0x4342),
                                               codes_h2(y, 0x4140), codes_h2(y, 0x4342)};
                        mma16816<MT>(oa[i], a, ph[0], ph[1]);
                        if constexpr (C::kTwoParts) mma16816<MT>(oa[i], a, pl[0], pl[1]);
                    }
                }
            }
        }
        __syncwarp();
        if (u_issue < u1) {
            issue(u_issue, s, 0u);
            ++u_issue;
        }
    }
    if (!aborted) {
        if (pb >= 0) finalize();
    } else {
        // A copy never completed: give the others a short bounded wait, then leave.
        for (long long v = u; v < u_issue; ++v) {
            const int sv = int((v - u0) % C::NS);
            mbar_wait_bounded(smem_addr(&bars[sv]), (parity >> sv) & 1u, kDrainLimitNs);
            parity ^= 1u << sv;
        }
    }
    if constexpr (ONE) {
        __syncthreads();
        constexpr int UT = UB * kBlockSize;
        const long long t0 = (long long)rank * one_nu / p.cluster * UT;
        const long long t1 = (long long)(rank + 1) * one_nu / p.cluster * UT;
        one_out<QT, D, G, M>(p, one_b, one_kvh, rank, s_ml, smem + kPrefixBytes, C::WARP_BYTES, C::STAGE,
                             int(t0), M == kMass ? int(min(t1, (long long)seq_len(p, one_b, false))) : 0);
        griddep_launch_dependents();   // not before: the next grid's CTAs would take its place
    }
}

// ------------------------------------------------------------------- join ---
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;

// out of segment (b, kvh) from its pieces wf .. wl (none: zeros): the float4
// items [slice, slice + 1) << lper of its G D / 4, by groups of one thread per
// item; group k merges pieces wf + k, wf + k + groups, ... and the groups merge
// in shared memory. Every thread of the CTA calls it with the same segment.
template <typename QT, int D, int G>
__device__ __forceinline__ void join_out(const Params& p, int b, int kvh, int wf, int wl, int slice,
                                         int lper, float2* s_ml, float4* s_o) {
    constexpr int Q = D / 4;
    static_assert(G * Q <= kJoinThreads, "threads cover the outputs");
    const long long seg = (long long)b * p.hkv + kvh;
    const int t = threadIdx.x, per = 1 << lper, groups = kJoinThreads >> lper;
    const int mine = t & (per - 1), item = (slice << lper) + mine, grp = t >> lper;
    const int h = item / Q, d4 = item - h * Q;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int w = wf + grp; w <= wl; w += groups) {
        const long long slot = seg + w;
        const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + (slot * G + h) * 2);
        fold(m, l, o, ml.x, ml.y, *reinterpret_cast<const float4*>(p.part_o + (slot * G + h) * D + d4 * 4));
    }
    if (groups > 1) {
        s_ml[t] = make_float2(m, l);
        s_o[t] = o;
        __syncthreads();
    }
    if (grp == 0) {
        const int used = min(groups, wl - wf + 1);
        for (int k = 1; k < used; ++k)
            fold(m, l, o, s_ml[(k << lper) + mine].x, s_ml[(k << lper) + mine].y, s_o[(k << lper) + mine]);
        const float2 v[2] = {make_float2(o.x, o.y), make_float2(o.z, o.w)};
        store_row<QT, 4>(p.out, ((long long)b * p.hq + kvh * G + h) * D + d4 * 4, v, reciprocal(l));
    }
}

// kMass: final (M, 1 / l) of segment seg's heads from its pieces wf .. wl, by
// N threads t = 0 .. N - 1 of which each 32 form a warp: every lane ends with
// the state of head lane % G over its warp's share of the pieces.
template <int G>
__device__ __forceinline__ void fold_ml(const Params& p, long long seg, int wf, int wl, int t, int n,
                                        float& m, float& l) {
    m = -INFINITY;
    l = 0.f;
#pragma unroll 4
    for (int w = wf + t / G; w <= wl; w += n / G) {
        const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + ((seg + w) * G + t % G) * 2);
        merge_ml(m, l, ml.x, ml.y);
    }
#pragma unroll
    for (int off = G; off < 32; off <<= 1) {
        const float m2 = __shfl_xor_sync(kFull, m, off), l2 = __shfl_xor_sync(kFull, l, off);
        merge_ml(m, l, m2, l2);
    }
}

// The last sequence b with P[b] <= x, by a warp: 32 places at a time.
__device__ __forceinline__ int find_sequence(const int* P, int batch, int x) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = batch;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const unsigned le = __ballot_sync(kFull, at < hi && P[at] <= x);   // lane 0 always
        lo += (31 - __clz(le)) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// kMass: the first mass_ctas CTAs share the batch's units in equal ranges and
// turn scores into weights. The further CTAs look after runs of segs_per_cta
// segments: those split over several workers are merged, those without units
// are zeroed (whole ones are written by the split kernel).
template <typename QT, int D, int G, int M, int UB>
__global__ void __launch_bounds__(kJoinThreads, 4) ctx_join_kernel(const Params p) {
    __shared__ float2 s_ml[kJoinThreads];
    __shared__ float4 s_o[kJoinThreads];
    griddep_wait();
    const int* P = p.ws_prefix;
    const long long U = (long long)P[p.batch] * p.hkv;
    const long long W = eff_workers(U, p.workers);
    if (M == kList || int(blockIdx.x) >= p.mass_ctas) {
        constexpr int LITEMS = (G == 1 ? 0 : G == 2 ? 1 : G == 4 ? 2 : 3) + (D == 64 ? 4 : 5);
        static_assert(1 << LITEMS == G * D / 4, "items of a segment's output");
        const int S = p.batch * p.hkv, x = int(blockIdx.x) - p.mass_ctas, slice = x & ((1 << p.lslices) - 1);
        const int seg0 = (x >> p.lslices) * p.segs_per_cta;
        const int lane = threadIdx.x & 31;
        for (int base = 0; base < p.segs_per_cta; base += 32) {
            // every warp checks the same 32 segments, one per lane
            bool todo_me = false;
            if (base + lane < p.segs_per_cta && seg0 + base + lane < S) {
                const int seg = seg0 + base + lane, b = seg / p.hkv, kvh = seg - b * p.hkv;
                const int nu = P[b + 1] - P[b];
                const long long uf = (long long)p.hkv * P[b] + (long long)kvh * nu;
                todo_me = nu == 0 || worker_of(uf, U, W) != worker_of(uf + nu - 1, U, W);
            }
            for (unsigned todo = __ballot_sync(kFull, todo_me); todo; todo &= todo - 1) {
                const int seg = seg0 + base + __ffs(todo) - 1, b = seg / p.hkv, kvh = seg - b * p.hkv;
                const int nu = P[b + 1] - P[b];
                const long long uf = (long long)p.hkv * P[b] + (long long)kvh * nu;
                const int wf = nu ? int(worker_of(uf, U, W)) : 0;
                const int wl = nu ? int(worker_of(uf + nu - 1, U, W)) : -1;
                join_out<QT, D, G>(p, b, kvh, wf, wl, slice, LITEMS - p.lslices, s_ml, s_o);
                __syncthreads();
            }
        }
    } else if constexpr (M == kMass) {
        // The CTA's share of the units. Inside one segment (long contexts, few
        // segments, many pieces) the whole CTA folds the pieces; otherwise every
        // warp goes through its own part, segment by segment.
        const long long n = p.mass_ctas, i = blockIdx.x;
        const long long c0 = i * U / n, c1 = (i + 1) * U / n;
        if (c0 >= c1) return;
        const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
        constexpr int UT = UB * kBlockSize;
        int b = find_sequence(P, p.batch, int(c0 / p.hkv)), kvh, nu = P[b + 1] - P[b], x0;
        {
            const int r = int(c0 - (long long)p.hkv * P[b]);
            kvh = r / nu;
            x0 = r - kvh * nu;
        }
        if (x0 + (c1 - c0) <= nu) {
            const long long seg = (long long)b * p.hkv + kvh, uf = c0 - x0;
            float m, l;
            fold_ml<G>(p, seg, int(worker_of(uf, U, W)), int(worker_of(uf + nu - 1, U, W)), t,
                       kJoinThreads, m, l);
            if (lane < G) s_ml[warp * G + lane] = make_float2(m, l);
            __syncthreads();
            float2 ml[G];
#pragma unroll
            for (int h = 0; h < G; ++h) {
                m = -INFINITY;
                l = 0.f;
#pragma unroll
                for (int w = 0; w < kJoinWarps; ++w) merge_ml(m, l, s_ml[w * G + h].x, s_ml[w * G + h].y);
                ml[h] = make_float2(m == -INFINITY ? 0.f : m, reciprocal(l));
            }
            weigh<G>(p, seg, x0 * UT, min(int(x0 + (c1 - c0)) * UT, seq_len(p, b, false)), t,
                     kJoinThreads, ml);
        } else {
            const long long u1 = c0 + (warp + 1) * (c1 - c0) / kJoinWarps;
            long long u = c0 + warp * (c1 - c0) / kJoinWarps;
            if (u < u1) {
                b = find_sequence(P, p.batch, int(u / p.hkv));
                nu = P[b + 1] - P[b];
                const int r = int(u - (long long)p.hkv * P[b]);
                kvh = r / nu;
                x0 = r - kvh * nu;
            }
            while (u < u1) {
                const int x1 = int(min((long long)nu, x0 + (u1 - u)));
                const long long seg = (long long)b * p.hkv + kvh, uf = u - x0;
                float m, l;
                fold_ml<G>(p, seg, int(worker_of(uf, U, W)), int(worker_of(uf + nu - 1, U, W)), lane,
                           32, m, l);
                const float top = m == -INFINITY ? 0.f : m, inv = reciprocal(l);
                float2 ml[G];
#pragma unroll
                for (int h = 0; h < G; ++h)
                    ml[h] = make_float2(__shfl_sync(kFull, top, h), __shfl_sync(kFull, inv, h));
                weigh<G>(p, seg, x0 * UT, min(x1 * UT, seq_len(p, b, false)), lane, 32, ml);
                u += x1 - x0;
                if (u >= u1) break;
                x0 = 0;            // the next segment with units
                if (++kvh == p.hkv) {
                    kvh = 0;
                    do {
                        ++b;
                        nu = P[b + 1] - P[b];
                    } while (nu == 0);
                }
            }
        }
    }
    griddep_launch_dependents();
}

// ------------------------------------------------------------------- host ---
inline bool is_aligned(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// A launch's configuration: programmatic dependent launch, clusters of `cluster` CTAs.
struct LaunchConfig {
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute attr[2];
    LaunchConfig(int grid, int threads, size_t smem, int cluster, cudaStream_t st) {
        c.gridDim = dim3(grid);
        c.blockDim = dim3(threads);
        c.dynamicSmemBytes = smem;
        c.stream = st;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = cluster;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        c.attrs = attr;
        c.numAttrs = cluster > 1 ? 2 : 1;
    }
};

struct Ops {
    int (*workers)(int dev);      // default worker warps on a device, 0 on an error
    cudaError_t (*run)(const Params&, int dev, cudaStream_t);
    cudaError_t (*run_one)(const Params&, int dev, cudaStream_t);   // p.cluster CTAs per segment
    int (*clusters)(int dev, int n);   // clusters of n ONE CTAs that a device holds at once
    int unit_blocks;
};

template <typename KV, typename QT, int D, int G, int M>
struct Impl {
    using C = Cfg<KV, QT, D, G>;
    // Resident worker warps of the device (looked up once), 2 CTAs per SM.
    static int workers(int dev) {
        static std::atomic<int> known[64];
        const bool keep = dev >= 0 && dev < 64;
        if (keep) {
            const int n = known[dev].load(std::memory_order_relaxed);
            if (n > 0) return n;
        }
        int sms = 0, blocks = 0;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        if (prepare() != cudaSuccess) return 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, ctx_split_kernel<KV, QT, D, G, M, false>,
                                                          C::THREADS, C::SMEM) != cudaSuccess)
            return 0;
        const int n = sms * (blocks < 2 ? blocks : 2) * C::WARPS;
        if (keep) known[dev].store(n, std::memory_order_relaxed);
        return n;
    }
    static cudaError_t prepare() {
        return cudaFuncSetAttribute(ctx_split_kernel<KV, QT, D, G, M, false>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    }
    // The kernel's leave for its shared memory is asked for once per device, and
    // again where a launch fails (a further context, a reset device).
    template <bool ONE>
    static cudaError_t launch(const Params& p, int grid, int dev, cudaStream_t st) {
        static std::atomic<unsigned long long> leave{0};
        constexpr int smem = ONE ? C::SMEM_ONE : C::SMEM;
        constexpr int threads = ONE ? 32 * kOneWarps : C::THREADS;
        const auto kernel = ctx_split_kernel<KV, QT, D, G, M, ONE>;
        LaunchConfig cfg(grid, threads, smem, ONE ? p.cluster : 1, st);
        const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
        if (leave.load(std::memory_order_relaxed) & bit) {
            if (cudaLaunchKernelEx(&cfg.c, kernel, p) == cudaSuccess) return cudaSuccess;
            cudaGetLastError();
        }
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg.c, kernel, p);
        if (e == cudaSuccess) leave.fetch_or(bit, std::memory_order_relaxed);
        return e;
    }
    static cudaError_t run(const Params& p, int dev, cudaStream_t st) {
        const cudaError_t e = launch<false>(p, 1 + (p.workers - 1) / C::WARPS, dev, st);
        if (e != cudaSuccess) return e;
        return launch_pdl(ctx_join_kernel<QT, D, G, M, C::UB>, dim3(p.mass_ctas + p.seg_ctas),
                          dim3(kJoinThreads), 0, st, p);
    }
    static cudaError_t run_one(const Params& p, int dev, cudaStream_t st) {
        return launch<true>(p, p.batch * p.hkv * p.cluster, dev, st);
    }
    // As many as 152 SMs hold CTAs, less what GPCs leave over (16 clusters of 8 do
    // not run side by side: 10.3 us instead of 5.7). Looked up once.
    static int clusters(int dev, int n) {
        static std::atomic<int> known[64][9];
        const bool keep = dev >= 0 && dev < 64;
        if (keep) {
            const int k = known[dev][n].load(std::memory_order_relaxed);
            if (k > 0) return k;
        }
        const auto kernel = ctx_split_kernel<KV, QT, D, G, M, true>;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_ONE) != cudaSuccess)
            return 0;
        LaunchConfig cfg(n, 32 * kOneWarps, C::SMEM_ONE, n, nullptr);
        int k = 0;
        if (cudaOccupancyMaxActiveClusters(&k, kernel, &cfg.c) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        if (keep) known[dev][n].store(k, std::memory_order_relaxed);
        return k;
    }
    static Ops ops() { return Ops{workers, run, run_one, clusters, C::UB}; }
};

template <int M, typename KV, typename QT, int D>
bool pick_g(int G, Ops* o) {
    switch (G) {
        case 1: *o = Impl<KV, QT, D, 1, M>::ops(); return true;
        case 2: *o = Impl<KV, QT, D, 2, M>::ops(); return true;
        case 4: *o = Impl<KV, QT, D, 4, M>::ops(); return true;
        case 8: *o = Impl<KV, QT, D, 8, M>::ops(); return true;
    }
    return false;
}

template <int M, typename KV, typename QT>
bool pick_d(int D, int G, Ops* o) {
    return D == 128 ? pick_g<M, KV, QT, 128>(G, o) : pick_g<M, KV, QT, 64>(G, o);
}

// INT8 caches: sparse_i8.cu, mass_i8.cu (units of their own, to compile side by side)
template <int M> bool pick_i8(pkv_dtype q, int D, int G, Ops* o);
template <> bool pick_i8<kList>(pkv_dtype q, int D, int G, Ops* o);
template <> bool pick_i8<kMass>(pkv_dtype q, int D, int G, Ops* o);

template <int M>
bool pick_ops(pkv_dtype kv, pkv_dtype q, int D, int G, Ops* o) {
    if (kv == PKV_BF16) return pick_d<M, BF16, BF16>(D, G, o);
    if (kv == PKV_F16) return pick_d<M, F16, F16>(D, G, o);
    return pick_i8<M>(q, D, G, o);
}

// How many CTAs per segment (a cluster) do a call of `segs` segments of up to
// `units` units (8 KB of K and V) each; 0: split over all workers and joined.
// A wave of CTAs takes 4 us, 1.5 more for a cluster's exchange, and 0.16 us (INT8:
// 0.235) per unit and CTA, whose 8 warps share them; split and join take 12 us
// and what the bytes cost at 7 TB/s. Alone and split, bf16 lists of head_dim 128:
// 8 of 128 blocks 7.5 and 13.2 us, of 2048 43.8 and 34.4; 128 of 128 25.5 and
// 31.8; 64 INT8 ones of 128 13.9 and 20.9. Only the most that a segment may hold
// is known here: split costs what is there, a CTA alone what the longest holds.
// So kMass expects half of the table's blocks to be in use, and nobody is left
// alone for more than 32 us or two waves.
template <int M>
int ctas_per_segment(const Ops& ops, int dev, bool i8, long long segs, long long units) {
    double best = std::min(32.0, 12.0 + (M == kMass ? 0.5 : 1.0) * double(segs) * double(units) / 850.0);
    int n = 0;
    if (segs > 304) return 0;
    for (int c = 1; c <= 8; c *= 2) {
        const long long room = c == 1 ? 152 : segs * c > 152 ? 0 : ops.clusters(dev, c);
        if (room == 0 || (c > 1 && segs > room)) break;
        const double wave = 4.0 + (c > 1 ? 1.5 : 0.0) + (i8 ? 0.235 : 0.16) * double(units) / c;
        const double t = double((segs + room - 1) / room) * wave;
        if (t < best) {
            best = t;
            n = c;
        }
    }
    return n;
}

struct Layout {
    size_t ml_off, o_off, scores_off, total;
};

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

inline Layout layout(int batch, int hkv, int G, int D, long long workers, long long score_tokens) {
    const size_t slots = size_t(batch) * hkv + size_t(workers);
    Layout l;
    l.ml_off = align256(sizeof(int32_t) * (size_t(batch) + 1));
    l.o_off = l.ml_off + align256(slots * G * 2 * sizeof(float));
    l.scores_off = l.o_off + align256(slots * G * D * sizeof(float));
    l.total = l.scores_off + align256(size_t(batch) * hkv * size_t(score_tokens) * G * sizeof(float));
    return l;
}

// Checks of sizes and types, shared by the size queries and the calls.
template <int M>
pkv_status check_sizes(const pkv_cache_desc* c, int batch, int hq, pkv_dtype q_dtype, Ops* ops,
                       int* G) {
    if (!c) return PKV_ERR_INVALID_ARG;
    if (c->num_blocks <= 0 || c->num_kv_heads <= 0 || c->head_dim <= 0) return PKV_ERR_INVALID_ARG;
    if (c->kv_dtype != PKV_F16 && c->kv_dtype != PKV_BF16 && c->kv_dtype != PKV_I8)
        return PKV_ERR_INVALID_ARG;
    if (q_dtype != PKV_F16 && q_dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
    if (batch < 0 || hq <= 0 || hq % c->num_kv_heads) return PKV_ERR_INVALID_ARG;
    if (c->block_size != kBlockSize || batch > kMaxBatch || c->num_kv_heads > 0xffff)
        return PKV_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (c->kv_dtype != PKV_I8 && q_dtype != c->kv_dtype) return PKV_ERR_INVALID_ARG;
    *G = hq / c->num_kv_heads;
    if ((long long)batch * c->num_kv_heads > 0x3fffffffLL) return PKV_ERR_UNSUPPORTED;
    return pick_ops<M>(c->kv_dtype, q_dtype, c->head_dim, *G, ops) ? PKV_OK : PKV_ERR_UNSUPPORTED;
}

template <int M>
size_t workspace_size(int batch, int hq, const pkv_cache_desc* c, int score_blocks, int num_parts) {
    Ops ops;
    int G = 0, dev = 0;
    const pkv_dtype qd = (c && c->kv_dtype == PKV_F16) ? PKV_F16 : PKV_BF16;
    if (check_sizes<M>(c, batch, hq, qd, &ops, &G) != PKV_OK || num_parts < 0) return 0;
    if (num_parts == 0 && cudaGetDevice(&dev) != cudaSuccess) return 0;
    const int workers = num_parts > 0 ? num_parts : ops.workers(dev);
    if (workers <= 0) return 0;
    return layout(batch, c->num_kv_heads, G, c->head_dim, workers,
                  (long long)score_blocks * kBlockSize).total;
}

// The pointers of p are set by the caller (all but the workspace's).
template <int M>
pkv_status run(Params p, pkv_dtype q_dtype, const pkv_cache_desc* c, int batch, int hq, int mb,
               float softmax_scale, void* workspace, size_t workspace_bytes, int num_parts,
               cudaStream_t stream, uint64_t wait_ns = kWaitLimitNs, int stall_worker = -1) {
    Ops ops;
    int G = 0, dev = 0;
    const pkv_status s = check_sizes<M>(c, batch, hq, q_dtype, &ops, &G);
    if (s != PKV_OK) return s;
    if (num_parts < 0) return PKV_ERR_INVALID_ARG;
    if (batch == 0) return PKV_OK;
    if (!p.q || !p.k_cache || !p.v_cache || !p.block_tables || !p.context_lens || !p.out)
        return PKV_ERR_INVALID_ARG;
    if (!is_aligned(p.q, 16) || !is_aligned(p.k_cache, 16) || !is_aligned(p.v_cache, 16) ||
        !is_aligned(p.out, 16) || !is_aligned(p.block_tables, 4) || !is_aligned(p.context_lens, 4) ||
        !is_aligned(p.status, 4))
        return PKV_ERR_INVALID_ARG;
    if (c->kv_dtype == PKV_I8 && (!p.k_scales || !p.v_scales || !is_aligned(p.k_scales, 4) ||
                                  !is_aligned(p.v_scales, 4)))
        return PKV_ERR_INVALID_ARG;
    if (mb <= 0 || mb > 0x7fffffff / kBlockSize) return PKV_ERR_INVALID_ARG;
    if ((long long)batch * mb > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;   // units are counted in 32 bits
    if (!(softmax_scale >= -3.0e38f && softmax_scale <= 3.0e38f)) return PKV_ERR_INVALID_ARG;
    if (num_parts == 0 && cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    const int workers = num_parts > 0 ? num_parts : ops.workers(dev);
    if (workers <= 0) return PKV_ERR_CUDA;
    const Layout l = layout(batch, c->num_kv_heads, G, c->head_dim, workers,
                            M == kMass ? (long long)mb * kBlockSize : 0);
    if (!workspace || workspace_bytes < l.total || !is_aligned(workspace, 256))
        return PKV_ERR_WORKSPACE;
    char* ws = static_cast<char*>(workspace);
    p.ws_prefix = reinterpret_cast<int32_t*>(ws);
    p.part_ml = reinterpret_cast<float*>(ws + l.ml_off);
    p.part_o = reinterpret_cast<float*>(ws + l.o_off);
    p.scores = reinterpret_cast<float*>(ws + l.scores_off);
    p.batch = batch; p.hq = hq; p.hkv = c->num_kv_heads; p.mb = mb; p.num_blocks = c->num_blocks;
    p.workers = workers;
    p.qscale = softmax_scale * kLog2e;
    p.wait_ns = wait_ns;
    p.stall_worker = stall_worker;
    // merging CTAs: up to 4 per SM (beside weighing CTAs, 128 KB of K and V each
    // and at most 4 per SM themselves: 2). More segments than that: runs of them
    // (4864 lists of 16 blocks: 107 us, with 2432 CTAs 111).
    const long long segs = (long long)batch * c->num_kv_heads;
    const long long most = M == kMass ? 304 : 608;
    p.keep_scores = M == kMass && l.total - l.scores_off <= (size_t(64) << 20);
    p.mass_ctas = 0;
    if (M == kMass) {
        const long long row = (long long)c->head_dim * (c->kv_dtype == PKV_I8 ? 1 : 2);
        const long long n = segs * mb * kBlockSize * row * 2 >> 17;
        p.mass_ctas = int(n < 1 ? 1 : n < 608 ? n : 608);
    }
    p.segs_per_cta = int((segs + most - 1) / most);
    // Few segments have many pieces: several CTAs share a segment's output, 128
    // bytes of a piece or more each (8 INT8 lists of 2048 blocks: 27.8 us, with
    // one CTA each 105; 192 of 192: 41.9, 43.9, and 43.9 with twice as many).
    p.lslices = 0;
    while ((segs << (p.lslices + 1)) <= most && (G * c->head_dim / 4 >> (p.lslices + 1)) >= 8) ++p.lslices;
    p.seg_ctas = int((segs + p.segs_per_cta - 1) / p.segs_per_cta) << p.lslices;
    if (num_parts > 0 && cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    const long long most_units = ((M == kList ? p.max_list : mb) + ops.unit_blocks - 1) / ops.unit_blocks;
    p.cluster = num_parts == 0 ? ctas_per_segment<M>(ops, dev, c->kv_dtype == PKV_I8, segs, most_units) : 0;
    const cudaError_t e = (p.cluster > 0 ? ops.run_one : ops.run)(p, dev, stream);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace ctx
}  // namespace pkv
