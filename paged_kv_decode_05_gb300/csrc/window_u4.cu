// Decode attention over a 4-bit cache (u4.cu has the format): the window mode of
// ctx_attn.cuh with a split kernel of its own.
//
// Mathematics. With codes c, pairs (s, lo) per row and q in fp16,
//   score_t = s_t <q, c_t> + lo_t sum(q),
//   out = sum_t (p_t s_t) c_t + sum_t p_t lo_t,   p = softmax,
// so only integers of 4 bits enter the products and a row's pair acts on its score
// and its weight. Products run on mma.sync m16n8k16 in fp16 with the group's heads in
// the N columns. A nibble in the lowest bits of an fp16 value is c 2^-24 exactly (a
// subnormal number), four bits further up c 2^-20: one AND turns two codes into
// operands, and powers of two make up for it, in q for scores, at the end for outputs.
//
// What bounds it: not the bytes (2.2 KB per block and kv head) but the instructions
// of a warp per block, and their latency. Therefore:
// * a warp feeds itself by 16-byte asynchronous copies, a whole warp to 512 bytes (of
//   bulk copies, one per tile and lane, the lanes come one by one: 103 instructions per
//   block without any arithmetic), with table entries fetched 30 units ahead into a ring
//   in shared memory;
// * the copies put rows where they are read without bank conflicts: K's rows so that a
//   lane's two tokens are neighbours, V's chunks swizzled for ldmatrix.trans, which
//   hands a lane four codes of two tokens in a word;
// * 16 warps per SM in 128 registers each.
// The units of one kv head are cut into ranges, and the warps of the hkv heads of a
// range sit side by side (ctx_attn.cuh).
//
// Measured (g = 4, D = 128, bf16 q, one GPU): 256 sequences of 128 to 4096 tokens 121 us
// for 0.60 GB (5.0 TB/s; the copies alone, without arithmetic, 104). From the INT8
// kernel's form: 203 us; codes without bias removal on one half, two-block units, 16
// warps: 151; subnormal operands, asynchronous copies, ldmatrix: 123; two stages instead
// of three: 121.
#include "ctx_attn.cuh"

namespace pkv {
namespace ctx {
namespace {

constexpr int kAhead = 30;                            // units fetched at a time
constexpr int kRing = 32;                             // entries: kAhead and the units not yet read

template <typename QT, int D, int G>
struct U4Cfg {
    static constexpr int ROW = D / 2, TILE = kBlockSize * ROW, PAIRS = kBlockSize * 4;
    static constexpr int STAGE = 4096;                // K tiles [UB], V tiles [UB]
    static constexpr int UB = STAGE / (2 * TILE);     // blocks per unit: 2, or 4 at head_dim 64
    static constexpr int NS = 2;                      // stages per warp (3: 124 us for 122)
    // P in two fp16 parts for an fp16 output, as over INT8: the second part takes the
    // columns that up to 4 heads leave free, or products of its own.
    static constexpr bool kTwo = std::is_same<QT, F16>::value, kSide = kTwo && G <= 4;
    static constexpr int COLS = kSide ? 2 * G : G;    // columns of P that hold something
    static constexpr int VIS = UB / 2;                // words of shown bits
    static constexpr int EW = UB == 2 ? 4 : 8;        // words of a ring entry
    static constexpr int OFF_PAIRS = NS * STAGE;      // [stage][block][K, V][16]
    static constexpr int OFF_RING = OFF_PAIRS + NS * 2 * UB * PAIRS;
    static constexpr int OFF_P = OFF_RING + kRing * EW * 4;
    static constexpr int PS = UB * 8 + 4;             // words (two tokens) of a row of P
    static constexpr int PROWS = kTwo ? 2 * G : G;
    static constexpr int WARP_BYTES = align_up(OFF_P + PROWS * PS * 4, 16);
    static constexpr int WARPS = kTwo && G == 8 ? 7 : 8;
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int SMEM = kPrefixBytes + WARPS * WARP_BYTES;
    static constexpr int SMEM_ONE = kPrefixBytes + kOneWarps * WARP_BYTES;
    static constexpr int NE = G == 1 ? 1 : 2;
    static_assert(UB == 2 || UB == 4, "two words of shown bits");
    static_assert(UB + VIS + 1 <= EW && kAhead + NS - 1 <= kRing, "ring");
    static_assert(2 * (SMEM + 1024) <= 233472, "two CTAs share an SM");
    static_assert(SMEM_ONE + 1024 <= 233472 && G * D * 4 <= STAGE, "a CTA per segment");
    static_assert((kOneWarps + 2) * G * 8 <= kPrefixBytes && NS >= 2, "(m, l) take the prefix's place");
    static_assert(WARPS <= kMaxWarps, "scan scratch");
};

// The codes at bits 0-3 of both halves as c 2^-24 in fp16, those at bits 4-7 as c 2^-20.
__device__ __forceinline__ uint32_t nibble_lo(uint32_t w) { return w & 0x000f000fu; }
__device__ __forceinline__ uint32_t nibble_hi(uint32_t w) { return w & 0x00f000f0u; }

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// Two fp32 additions in one operation.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 c, a, b;\n\tmov.b64 {%0, %1}, c;}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

template <typename QT, int D, int G, bool ONE>
__global__ void __launch_bounds__(ONE ? 32 * kOneWarps : U4Cfg<QT, D, G>::THREADS, ONE ? 1 : 2)
u4_split_kernel(const Params p) {
    using C = U4Cfg<QT, D, G>;
    constexpr int UB = C::UB, NT = D / 16;
    extern __shared__ __align__(128) unsigned char smem[];
    int* warp_tot = reinterpret_cast<int*>(smem);
    int* prefix = warp_tot + kMaxWarps;
    float2* s_ml = reinterpret_cast<float2*>(smem);   // ONE: [kOneWarps][G]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * (ONE ? kOneWarps : C::WARPS) + warp;
    int one_b = 0, one_nu = 0, rank = 0, kvh;
    long long u0, slot0 = 0;
    int units;                                        // of this worker: u0, u0 + 1, ...
    griddep_wait();
    if constexpr (ONE) {
        const int seg = int(blockIdx.x) / p.cluster;
        rank = int(blockIdx.x) - seg * p.cluster;
        one_b = seg / p.hkv;
        kvh = seg - one_b * p.hkv;
        one_nu = seq_units<kWindow, UB>(p, one_b, kvh == 0 && rank == 0 && threadIdx.x == 0);
        const int share = rank * kOneWarps + warp, shares = p.cluster * kOneWarps;
        u0 = (long long)share * one_nu / shares;
        units = int((long long)(share + 1) * one_nu / shares - u0);
        if (lane < G) s_ml[warp * G + lane] = make_float2(-INFINITY, 0.f);
    } else {
        griddep_launch_dependents();
        build_prefix<kWindow, UB, C::THREADS>(p, warp_tot, prefix);
        const long long U = prefix[prefix_chunks(p.batch)];      // units of one kv head
        const long long W = eff_workers(U, ranges(p.workers, p.hkv)), r = w / p.hkv;
        if (r >= W || U == 0) return;
        u0 = r * U / W;
        units = int((r + 1) * U / W - u0);
        kvh = int(w - r * p.hkv);
        slot0 = kvh * (p.batch + W) + r;              // + sequence
    }

    unsigned char* region = smem + kPrefixBytes + warp * C::WARP_BYTES;
    uint32_t* ring = reinterpret_cast<uint32_t*>(region + C::OFF_RING);
    uint32_t* pw = reinterpret_cast<uint32_t*>(region + C::OFF_P);
    // ---- producer. A ring entry: the physical blocks (-1: none), the bits of their
    // shown tokens, the sequence and flags: first and last unit of the segment << 29
    // and << 30.
    struct Entry {
        int blk[UB];
        uint32_t vis[C::VIS], tag;
    };
    auto fetch = [&](int from) {
        Entry a;
        const int i0 = from + lane;
        a.tag = 0u;
#pragma unroll
        for (int i = 0; i < UB; ++i) a.blk[i] = -1;
#pragma unroll
        for (int i = 0; i < C::VIS; ++i) a.vis[i] = 0u;
        if (lane < kAhead && i0 < units) {
            int b = one_b, j = int(u0) + i0, nu = one_nu, zero;
            if constexpr (!ONE) find_unit<kWindow, UB>(u0 + i0, prefix, p, b, zero, j, nu);
            const int L = seq_len(p, b, false);
            const Shown see = shown(p, L);
            const int entries = (L + kBlockSize - 1) / kBlockSize - see.skip;
            a.tag = b | (j == 0 ? 1 << 29 : 0) | (j == nu - 1 ? 1 << 30 : 0);
#pragma unroll
            for (int i = 0; i < UB; ++i) {
                const int e = UB * j + i;
                if (e >= entries) continue;
                const int id = e + (e >= see.lead ? see.skip : 0);
                const int blk = __ldg(p.block_tables + (long long)b * p.mb + id);
                if (unsigned(blk) >= unsigned(p.num_blocks)) {
                    flag_status(p.status, PKV_DEV_BAD_BLOCK);
                    continue;
                }
                a.blk[i] = blk;
                a.vis[i / 2] |= shown_bits(see, L, id * kBlockSize) << (16 * (i & 1));
            }
        }
        return a;
    };
    auto put = [&](int from, const Entry& a) {
        if (lane >= kAhead) return;
        uint32_t* e = ring + ((from + lane) & (kRing - 1)) * C::EW;
        if constexpr (UB == 2) {
            *reinterpret_cast<uint4*>(e) = make_uint4(a.blk[0], a.blk[1], a.vis[0], a.tag);
        } else {
            *reinterpret_cast<uint4*>(e) = make_uint4(a.blk[0], a.blk[1], a.blk[2], a.blk[UB - 1]);
            *reinterpret_cast<uint4*>(e + 4) = make_uint4(a.vis[0], a.vis[C::VIS - 1], a.tag, 0u);
        }
    };
    constexpr int TAG = UB == 2 ? 3 : 6, SHOW = UB;   // words of an entry
    put(0, fetch(0));
    int limit = kAhead;
    Entry ahead = fetch(limit);
    __syncwarp();

    // A lane's part of a tile's copies: 16 bytes of row t, and for D = 128 of row t + 8.
    // K's row of token t lies at t / 2 + 8 (t % 2), so that rows gq, gq + 8 of a lane
    // are tokens 2 gq, 2 gq + 1; V's chunks change places from row to row so that the 8
    // rows of a matrix lie in different banks.
    constexpr int CH = C::ROW / 16;                   // chunks per row: 4 or 2
    const int t0 = lane / CH, c0 = lane % CH;
    const uint32_t k_to = (t0 / 2 + 8 * (t0 & 1)) * C::ROW + 16 * c0;
    const uint32_t v_to = UB * C::TILE + t0 * C::ROW + 16 * (c0 ^ (CH == 4 ? t0 >> 1 & 3 : t0 >> 2 & 1));
    const char* k_from = static_cast<const char*>(p.k_cache) + (long long)kvh * C::TILE + 16 * lane;
    const char* v_from = static_cast<const char*>(p.v_cache) + (long long)kvh * C::TILE + 16 * lane;
    const long long tile_step = (long long)p.hkv * C::TILE;      // between blocks
    // and 16 bytes of the pairs of K or V of block lane / 8
    const char* p_from = reinterpret_cast<const char*>(lane & 4 ? p.v_scales : p.k_scales) +
                         (long long)kvh * C::PAIRS + 16 * (lane & 3);
    const int pair_step = p.hkv * C::PAIRS;
    const uint32_t to0 = smem_addr(region);

    auto issue = [&](int i, int s) {
        if (i == limit) {
            // overwrites units limit - 32 and before; the NS - 1 units not yet read stay
            put(limit, ahead);
            limit += kAhead;
            __syncwarp();
            ahead = fetch(limit);
        }
        const uint32_t* e = ring + (i & (kRing - 1)) * C::EW;
        const uint32_t to = to0 + s * C::STAGE, tag = e[TAG];
#pragma unroll
        for (int bi = 0; bi < UB; ++bi) {
            const int blk = int(e[bi]);
            if (blk < 0) continue;
            const long long off = blk * tile_step;
            cp_async_16(to + k_to + bi * C::TILE, k_from + off);
            cp_async_16(to + v_to + bi * C::TILE, v_from + off);
            if constexpr (CH == 4) {                  // rows t + 8
                cp_async_16(to + k_to + 4 * C::ROW + bi * C::TILE, k_from + off + 512);
                cp_async_16(to + v_to + 8 * C::ROW + bi * C::TILE, v_from + off + 512);
            }
        }
        const int of = lane < 8 * UB ? int(e[lane / 8]) : -1;
        if (of >= 0) cp_async_16(to0 + C::OFF_PAIRS + (s * 8 * UB + lane) * 16, p_from + (long long)of * pair_step);
        if ((i == 0 || (tag >> 29 & 1u)) && lane < G * D / 32)   // the piece's q rows into L2
            asm volatile("prefetch.global.L2 [%0];" ::"l"(
                static_cast<const uint16_t*>(p.q) + ((long long)(tag & 0x1fffu) * p.hq + kvh * G) * D + 32 * lane));
    };

    // ---- consumer. Lane (gq, tq) = (lane / 4, lane % 4) holds the scores of tokens
    // 2 gq, 2 gq + 1 of a block for columns 2tq, 2tq + 1 (heads; kSide: column G + h is
    // head h again, for P's second part), and accumulates dims 32 c + 4 gq + [0, 4) of O:
    // m-tiles 2c, 2c + 1 have the first and second two, the even in row gq.
    const int gq = lane >> 2, tq = lane & 3;
    uint32_t qb[NT][2];
    float2 qs = make_float2(p.qscale, p.qscale);      // score factors of the two columns
    float2 qsum = {}, losum = {};                     // sum(q) times the factor, sum of P lo
    float2 m = {}, lsum = {};
    float oa[NT][4];
    int pb = -1;
    bool first_seen = false, last_seen = false;
    // P carries s into fp16, O is kept in units of 2^vexp, chosen from the piece's
    // first scales so that a weight of 1 sits near 2^13 and raised when a later scale
    // would pass 2^14. vmul = 2^-vexp, 0 until chosen.
    int vexp = 0;
    float vmul = 0.f;

    auto finalize = [&]() {
        float lh[2] = {lsum.x, lsum.y}, lo[2] = {losum.x, losum.y};
        const float up = ldexpf(1.f, vexp);
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                lh[e] += __shfl_xor_sync(kFull, lh[e], off);
                lo[e] += __shfl_xor_sync(kFull, lo[e], off);
            }
        if constexpr (C::kSide) {                     // the second part's columns, G to the right
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int r = 0; r < 4; r += 2) {
                    if constexpr (G == 1) {
                        oa[i][r] += oa[i][r + 1];
                    } else {
                        oa[i][r] += __shfl_xor_sync(kFull, oa[i][r], G / 2);
                        oa[i][r + 1] += __shfl_xor_sync(kFull, oa[i][r + 1], G / 2);
                    }
                }
        }
#pragma unroll
        for (int e = 0; e < C::NE; ++e) {
            const int h = 2 * tq + e;
            if (h >= G) continue;
            float4 v[NT / 2];
#pragma unroll
            for (int c = 0; c < NT / 2; ++c)          // 2^24 first: 2^vexp may be 2^113
                v[c] = make_float4(fmaf(oa[2 * c][e] * 0x1p24f, up, lo[e]), fmaf(oa[2 * c][2 + e] * 0x1p20f, up, lo[e]),
                                   fmaf(oa[2 * c + 1][e] * 0x1p24f, up, lo[e]),
                                   fmaf(oa[2 * c + 1][2 + e] * 0x1p20f, up, lo[e]));
            const float mh = e ? m.y : m.x;
            if (!ONE && first_seen && last_seen) {
                const float inv = reciprocal(lh[e]);
#pragma unroll
                for (int c = 0; c < NT / 2; ++c) {
                    const float2 x[2] = {make_float2(v[c].x, v[c].y), make_float2(v[c].z, v[c].w)};
                    store_row<QT, 4>(p.out, ((long long)pb * p.hq + kvh * G + h) * D + 32 * c + 4 * gq, x, inv);
                }
                continue;
            }
            const long long slot = slot0 + pb;
            float* dst = ONE ? reinterpret_cast<float*>(region) + h * D     // its first stage is free
                             : p.part_o + (slot * G + h) * D;
#pragma unroll
            for (int c = 0; c < NT / 2; ++c) *reinterpret_cast<float4*>(dst + 32 * c + 4 * gq) = v[c];
            if (gq == 0) {
                if constexpr (ONE) s_ml[warp * G + h] = make_float2(mh, lh[e]);
                else *reinterpret_cast<float2*>(p.part_ml + (slot * G + h) * 2) = make_float2(mh, lh[e]);
            }
        }
    };

#pragma unroll
    for (int s = 0; s < C::NS; ++s) {
        if (s < units) issue(s, s);
        cp_async_commit();
    }
    for (int i = 0, s = 0; i < units; ++i, s = (s + 1 == C::NS) ? 0 : s + 1) {
        cp_async_wait<C::NS - 1>();                   // this lane's copies of unit i
        __syncwarp();                                 // and the others'
        const uint32_t* e = ring + (i & (kRing - 1)) * C::EW;
        const uint32_t tag = e[TAG], vis0 = e[SHOW], vis1 = e[SHOW + C::VIS - 1];
        const bool first = (tag >> 29 & 1u) != 0;
        if (i == 0 || first) {                        // first unit of a new piece
            if (pb >= 0) finalize();
            pb = tag & 0x1fffu;
            first_seen = first;
            const uint16_t* qs16 = static_cast<const uint16_t*>(p.q) + ((long long)pb * p.hq + kvh * G) * D;
            // q^T as the B operand: k-steps 2c, 2c + 1 of lane tq read dims D/4 tq + 8c
            // + [0, 8) in the order 0 4 1 5 and 2 6 3 7 that a word of codes falls into
            float amax = 0.f;
#pragma unroll
            for (int c = 0; c < NT / 2; ++c) {
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (gq < C::COLS) x = __ldg(reinterpret_cast<const uint4*>(qs16 + gq % G * D + D / 4 * tq + 8 * c));
                qb[2 * c][0] = __byte_perm(x.x, x.z, 0x5410);
                qb[2 * c][1] = __byte_perm(x.x, x.z, 0x7632);
                qb[2 * c + 1][0] = __byte_perm(x.y, x.w, 0x5410);
                qb[2 * c + 1][1] = __byte_perm(x.y, x.w, 0x7632);
            }
            // into fp16's range by a power of two, the channels at bits 4-7 of their half
            // by a 16th of it; a head's dims lie in lanes 4 gq + [0, 4)
#pragma unroll
            for (int kk = 0; kk < NT; ++kk)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2 f = unpack2(QT{}, qb[kk][k]);
                    amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
            amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
            const float2 fit = fit_half(amax);
            float sum = 0.f;
#pragma unroll
            for (int kk = 0; kk < NT; ++kk) {
                const float2 f = unpack2(QT{}, qb[kk][0]), h = unpack2(QT{}, qb[kk][1]);
                const float2 f2 = make_float2(f.x * fit.x, f.y * fit.x), h2 = make_float2(h.x * fit.x, h.y * fit.x);
                sum += (f2.x + f2.y) + (h2.x + h2.y);
                qb[kk][0] = pack2<F16>(f2.x, f2.y);
                qb[kk][1] = pack2<F16>(h2.x * 0.0625f, h2.y * 0.0625f);
            }
            sum += __shfl_xor_sync(kFull, sum, 1);
            sum += __shfl_xor_sync(kFull, sum, 2);
            const int a = 8 * tq, b = 8 * tq + 4;     // lanes that hold columns 2tq, 2tq + 1
            qs = make_float2(p.qscale * __shfl_sync(kFull, fit.y, a), p.qscale * __shfl_sync(kFull, fit.y, b));
            qsum = make_float2(qs.x * __shfl_sync(kFull, sum, a), qs.y * __shfl_sync(kFull, sum, b));
            losum = lsum = make_float2(0.f, 0.f);
            m = make_float2(-INFINITY, -INFINITY);
#pragma unroll
            for (int k = 0; k < NT; ++k) oa[k][0] = oa[k][1] = oa[k][2] = oa[k][3] = 0.f;
            vexp = 0;
            vmul = 0.f;
        }
        last_seen = (tag >> 30 & 1u) != 0;

        if (vis0 | vis1) {
            constexpr int KW = D / 32;                // words of codes per lane and row of K
            const unsigned char* kt = region + s * C::STAGE;
            const uint32_t vt = to0 + s * C::STAGE + UB * C::TILE;
            const uint32_t* pairs = reinterpret_cast<const uint32_t*>(region + C::OFF_PAIRS) + s * 2 * UB * kBlockSize;
            // ---- scores in log2 units
            float2 sc[UB][2], vp[UB][2];              // of tokens 2 gq, 2 gq + 1; (s, lo) of their V rows
#pragma unroll
            for (int bi = 0; bi < UB; ++bi) {
                float acc[2][4] = {};                 // two chains of products
                const unsigned char* kb = kt + bi * C::TILE + gq * C::ROW + 4 * KW * tq;
                uint32_t x[2][KW];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    if constexpr (KW == 4) {
                        const uint4 y = *reinterpret_cast<const uint4*>(kb + 8 * r * C::ROW);
                        x[r][0] = y.x; x[r][1] = y.y; x[r][2] = y.z; x[r][3] = y.w;
                    } else {
                        const uint2 y = *reinterpret_cast<const uint2*>(kb + 8 * r * C::ROW);
                        x[r][0] = y.x; x[r][1] = y.y;
                    }
                }
#pragma unroll
                for (int c = 0; c < KW; ++c)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t x0 = x[0][c] >> (8 * k), x1 = x[1][c] >> (8 * k);
                        const uint32_t a[4] = {nibble_lo(x0), nibble_lo(x1), nibble_hi(x0), nibble_hi(x1)};
                        mma16816<F16>(acc[k], a, qb[2 * c + k][0], qb[2 * c + k][1]);
                    }
                const uint2 kp2 = *reinterpret_cast<const uint2*>(pairs + 2 * bi * kBlockSize + 2 * gq);
                const uint2 vp2 = *reinterpret_cast<const uint2*>(pairs + (2 * bi + 1) * kBlockSize + 2 * gq);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float2 kp = unpack2(QT{}, r ? kp2.y : kp2.x);
                    vp[bi][r] = unpack2(QT{}, r ? vp2.y : vp2.x);
                    const float2 d = add2(make_float2(acc[0][2 * r], acc[0][2 * r + 1]),
                                          make_float2(acc[1][2 * r], acc[1][2 * r + 1]));
                    const float ks = kp.x * 0x1p24f;  // not on qs, which may be near 2^113
                    sc[bi][r].x = fmaf(d.x, ks * qs.x, qsum.x * kp.y);
                    sc[bi][r].y = fmaf(d.y, ks * qs.y, qsum.y * kp.y);
                }
            }
            if ((vis0 & vis1) != 0xffffffffu) {       // hidden tokens: their pairs may hold anything
#pragma unroll
                for (int bi = 0; bi < UB; ++bi)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        if (!(((bi < 2 ? vis0 : vis1) >> (16 * (bi & 1) + 2 * gq + r)) & 1u)) {
                            sc[bi][r] = make_float2(-INFINITY, -INFINITY);
                            vp[bi][r] = make_float2(0.f, 0.f);
                        }
            }
            // ---- P's exponent
            float vmax = vp[0][0].x;
#pragma unroll
            for (int k = 1; k < 2 * UB; ++k) vmax = fmaxf(vmax, vp[k / 2][k % 2].x);
            if (__any_sync(kFull, vmax > 0.f && (vmul == 0.f || vmax * vmul >= 16384.f))) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) vmax = fmaxf(vmax, __shfl_xor_sync(kFull, vmax, off));
                int ex;
                frexpf(vmax, &ex);                    // vmax < 2^ex
                const int nexp = min(max(ex - 13, -126), 126);
                if (vmul != 0.f) {
                    const float r = ldexpf(1.f, vexp - nexp);
#pragma unroll
                    for (int k = 0; k < NT; ++k) {
                        oa[k][0] *= r; oa[k][1] *= r; oa[k][2] *= r; oa[k][3] *= r;
                    }
                }
                vexp = nexp;
                vmul = ldexpf(1.f, -nexp);
            }
            // ---- running maximum and sum; P into shared memory, two tokens of a column to a
            // word, those that a lane reads side by side
            float2 mx = sc[0][0];
#pragma unroll
            for (int k = 1; k < 2 * UB; ++k) {
                mx.x = fmaxf(mx.x, sc[k / 2][k % 2].x);
                mx.y = fmaxf(mx.y, sc[k / 2][k % 2].y);
            }
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                mx.x = fmaxf(mx.x, __shfl_xor_sync(kFull, mx.x, off));
                mx.y = fmaxf(mx.y, __shfl_xor_sync(kFull, mx.y, off));
            }
            mx.x = fmaxf(m.x, mx.x);
            mx.y = fmaxf(m.y, mx.y);
            const float2 base = make_float2(mx.x == -INFINITY ? 0.f : -mx.x, mx.y == -INFINITY ? 0.f : -mx.y);
            if (__any_sync(kFull, mx.x != m.x || mx.y != m.y)) {
                const float ax = mx.x == -INFINITY ? 1.f : fast_exp2(m.x - mx.x);
                const float ay = mx.y == -INFINITY ? 1.f : fast_exp2(m.y - mx.y);
                m = mx;
                lsum.x *= ax; lsum.y *= ay;
                losum.x *= ax; losum.y *= ay;
#pragma unroll
                for (int k = 0; k < NT; ++k) {
                    oa[k][0] *= ax; oa[k][1] *= ay;
                    oa[k][2] *= ax; oa[k][3] *= ay;
                }
            }
            const int at = 2 * (gq & 3) + (gq >> 2);
#pragma unroll
            for (int bi = 0; bi < UB; ++bi) {
                float2 wt[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float2 x = add2(sc[bi][r], base);
                    const float2 ex = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                    lsum = add2(lsum, ex);
                    const float v = vp[bi][r].x * vmul;
                    losum.x = fmaf(ex.x, vp[bi][r].y, losum.x);
                    losum.y = fmaf(ex.y, vp[bi][r].y, losum.y);
                    wt[r] = make_float2(ex.x * v, ex.y * v);
                }
#pragma unroll
                for (int e2 = 0; e2 < 2; ++e2) {
                    const int col = 2 * tq + e2;
                    const float a = e2 ? wt[0].y : wt[0].x, b = e2 ? wt[1].y : wt[1].x;
                    uint32_t hi = pack2<F16>(a, b), lo = 0u;
                    if constexpr (C::kTwo) {
                        const float2 h = unpack2(F16{}, hi);
                        lo = pack2<F16>(a - h.x, b - h.y);
                        if (C::kSide && col >= G) hi = lo;
                    }
                    if (col < C::COLS) {
                        pw[col * C::PS + 8 * bi + at] = hi;
                        if constexpr (C::kTwo && !C::kSide) pw[(G + col) * C::PS + 8 * bi + at] = lo;
                    }
                }
            }
            __syncwarp();
            // ---- O^T += V^T P^T. A word of an 8x8 matrix of 16-bit pieces, transposed, holds
            // four codes of tokens 2tq, 2tq + 1 (+ 8); matrices: tokens 0-7 and 8-15 of
            // chunks c and c + 1.
            const int tok = lane & 15, ch = lane >> 4;
            const uint32_t vrow = vt + tok * C::ROW, vsw = CH == 4 ? tok >> 1 & 3 : tok >> 2 & 1;
#pragma unroll
            for (int bi = 0; bi < UB; ++bi) {
                uint2 ph = make_uint2(0u, 0u), pl = ph;
                if (gq < C::COLS) {
                    ph = *reinterpret_cast<const uint2*>(pw + gq * C::PS + 8 * bi + 2 * tq);
                    if constexpr (C::kTwo && !C::kSide)
                        pl = *reinterpret_cast<const uint2*>(pw + (G + gq) * C::PS + 8 * bi + 2 * tq);
                }
#pragma unroll
                for (int c = 0; c < CH; c += 2) {
                    uint32_t x[4];
                    ldsm_x4_trans(vrow + bi * C::TILE + (((c + ch) ^ vsw) << 4), x);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {     // chunk c + k / 2, first or second two dims
                        const uint32_t y0 = x[k & 2] >> (8 * (k & 1)), y1 = x[(k & 2) + 1] >> (8 * (k & 1));
                        const uint32_t a[4] = {nibble_lo(y0), nibble_hi(y0), nibble_lo(y1), nibble_hi(y1)};
                        mma16816<F16>(oa[2 * c + k], a, ph.x, ph.y);
                        if constexpr (C::kTwo && !C::kSide) mma16816<F16>(oa[2 * c + k], a, pl.x, pl.y);
                    }
                }
            }
        }
        __syncwarp();
        if (i + C::NS < units) issue(i + C::NS, s);
        cp_async_commit();
    }
    if (pb >= 0) finalize();
    if constexpr (ONE) {
        __syncthreads();
        one_out<QT, D, G, kWindow>(p, one_b, kvh, rank, s_ml, smem + kPrefixBytes, C::WARP_BYTES, C::STAGE, 0, 0);
        griddep_launch_dependents();   // not before: the next grid's CTAs would take its place
    }
}

template <typename QT, int D, int G>
struct U4Kernels {
    using C = U4Cfg<QT, D, G>;
    template <bool ONE>
    static auto split() { return u4_split_kernel<QT, D, G, ONE>; }
    static auto join() { return ctx_join_kernel<QT, D, G, kWindow, C::UB>; }
};

template <typename QT, int D>
bool pick_u4(int G, Ops* o) {
    switch (G) {
        case 1: *o = Impl<U4Kernels<QT, D, 1>>::ops(); return true;
        case 2: *o = Impl<U4Kernels<QT, D, 2>>::ops(); return true;
        case 4: *o = Impl<U4Kernels<QT, D, 4>>::ops(); return true;
        case 8: *o = Impl<U4Kernels<QT, D, 8>>::ops(); return true;
    }
    return false;
}

}  // namespace

bool pick_window_u4(pkv_dtype q, int D, int G, Ops* o) {
    if (q == PKV_BF16) return D == 128 ? pick_u4<BF16, 128>(G, o) : pick_u4<BF16, 64>(G, o);
    return D == 128 ? pick_u4<F16, 128>(G, o) : pick_u4<F16, 64>(G, o);
}

}  // namespace ctx
}  // namespace pkv
