// Multi-query paged attention: the tcgen05 kernel for long query runs (mq.cu
// instantiates it).
#pragma once

#include "mq_split.cuh"
#include "tc.cuh"

namespace pkv {

using TcLaunch = cudaError_t (*)(const CUtensorMap&, const CUtensorMap&, const MqParams&, int,
                                 cudaStream_t);

namespace {

// ------------------------------------------------- tcgen05 row-tile kernel ---
// Long query runs (prefill chunks): a CTA owns two tiles of 128 rows of one
// (sequence, kv head), rows = (query, head) pairs, and walks their visible
// tokens in chunks of 64 (four blocks) on the 5th-generation tensor cores:
//   S = Q K^T      tcgen05.mma kind::f16, M = 128, N = 64, K = D, fp32 in TMEM
//   softmax        one thread per row reads its S row from TMEM (no shuffles)
//   O += P V       tcgen05.mma, M = 128, N = D, K = 64; P from tensor memory
//                  (hi + lo 16-bit parts, written by the softmax over its own
//                  S buffer), V read MN-major straight from its TMA tile; O
//                  stays in TMEM for the whole tile.
// Warp 0 produces (TMA of K/V chunks into NSTG stages), warp 1 issues the MMAs
// and owns the TMEM allocation, warps 2-9 run the softmax and the epilogue
// (four warps per tile, one thread per row).
// Operands in shared memory use the 128-byte swizzle (TMA writes K/V that way;
// Q is written by threads in the same pattern). O is rescaled only when
// a row's running maximum grows by more than 2^8 (then exactly); in between P
// is taken against the older maximum, and O and l always share it.

constexpr int kTcChunk = 64;       // tokens per chunk
constexpr int kTcStages = 5;

// The two tiles (rows of tiles 2u and 2u + 1) share every K/V chunk: while
// one tile's softmax runs, the tensor core works on the other tile's S or
// P.V. Warps 2-5 are tile 0's softmax, warps 6-9 tile 1's. TMEM (512
// columns): S buffers of tile x at 128 x + 64 (c % 2), O of tile x at
// 256 + 128 x. P of chunk c replaces S of chunk c in its buffer (hi in the
// first 32 columns, lo in the next 32, two 16-bit values per column): the
// MMAs of a thread run in issue order, so the P.V of chunk c reads it before
// the S of chunk c + 2 overwrites the buffer, and the softmax of chunk c
// writes it while the P.V of chunk c - 1 still runs (it waits for that P.V
// only before touching O).
constexpr int kTcThreads = 64 + 2 * kTcRows;

template <int D>
struct TcCfg {
    static constexpr int NH = D / 64;
    static constexpr int HALF = kTcChunk * 128;
    static constexpr int KV_STAGE = 2 * NH * HALF;
    static constexpr int QHALF = kTcRows * 128;
    static constexpr int QTILE = NH * QHALF;
    static constexpr int OFF_Q = 0;                                  // tile x at OFF_Q + x QTILE
    static constexpr int OFF_KV = OFF_Q + 2 * QTILE;
    static constexpr int OFF_BAR = OFF_KV + kTcStages * KV_STAGE;
    // kv_full[S], kv_empty[S], s_full[2 tiles][2], p_full[2], o_done[2], drain
    static constexpr int NBAR = 2 * kTcStages + 9;
    static constexpr int OFF_MASK = OFF_BAR + NBAR * 8;
    static constexpr int OFF_MISC = OFF_MASK + kTcStages * 4;
    static constexpr int BYTES = OFF_MISC + 16 + 1024;
    static constexpr int TMEM_COLS = 512;
    static_assert(D == 64 || D == 128, "head_dim");
    static_assert(OFF_KV % 1024 == 0, "swizzle atoms");
};

template <typename KV, int D, int G>
__global__ void __launch_bounds__(kTcThreads, 1)
mq_tc_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
              const MqParams p) {
    using C = TcCfg<D>;
    constexpr int QPT = kTcRows / G;   // queries per tile
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* kv_full = bars;
    uint64_t* kv_empty = bars + kTcStages;
    uint64_t* s_full = bars + 2 * kTcStages;          // [tile][buffer]
    uint64_t* p_full = bars + 2 * kTcStages + 4;      // [tile]
    uint64_t* o_done = bars + 2 * kTcStages + 6;      // [tile]
    uint64_t* drain = bars + 2 * kTcStages + 8;
    int* smask = reinterpret_cast<int*>(smem + C::OFF_MASK);
    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    griddep_wait();
    griddep_launch_dependents();
    // unit: (sequence b, kv head, tile pair u); heavier (later) pairs first
    const int tpair = (p.tmax + 1) / 2;
    const long long unit = blockIdx.x;
    const int u = tpair - 1 - int(unit % tpair);
    const int kvh = int((unit / tpair) % p.hkv);
    const int b = int(unit / ((long long)tpair * p.hkv));
    int n, L;
    bool bad;
    seq_shape_raw(p.cu_q, p.context_lens, b, p.mb, p.max_q, n, L, bad);
    if (bad && threadIdx.x == 0 && kvh == 0 && u == 0) flag_status(p.status, PKV_DEV_BAD_LENGTH);
    const int q00 = 2 * u * QPT;                           // first query of tile 0
    if (q00 >= n) return;   // the whole CTA leaves before any allocation
    const bool two = q00 + QPT < n;                         // tile 1 holds queries too
    const int cu = p.cu_q[b];
    const int q_last = min(n, q00 + (two ? 2 : 1) * QPT) - 1;
    const int pos_max = L - n + q_last;                    // last token any row may see
    const int nch = (pos_max + 1 + kTcChunk - 1) / kTcChunk;
    const int jmax = pos_max / kBlockSize;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NBAR; ++i) mbar_init(smem_addr(&bars[i]), 1);
        fence_mbar_init();
        misc[1] = 0u;
    }
    for (int i = threadIdx.x; i < kTcStages * C::KV_STAGE / 16; i += kTcThreads) {
        const int s = i / (C::KV_STAGE / 16), off = i % (C::KV_STAGE / 16);
        if (off >= C::NH * C::HALF / 16)
            reinterpret_cast<uint4*>(smem + C::OFF_KV + s * C::KV_STAGE)[off] = make_uint4(0u, 0u, 0u, 0u);
    }
    // both Q tiles (query q00 + R / G, head R % G for R in 0 .. 255), zero past
    // the sequence, 128-byte-swizzled K-major
    for (int i = threadIdx.x; i < 2 * kTcRows * (D / 8); i += kTcThreads) {
        const int R = i / (D / 8), c16 = i % (D / 8);
        const int x = R / kTcRows, r = R % kTcRows;
        const int qi = q00 + R / G, h = R % G;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (qi < n)
            v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                ((long long)(cu + qi) * p.hq + kvh * G + h) * D + c16 * 8);
        const int half = c16 / 8, c = c16 % 8;
        *reinterpret_cast<uint4*>(smem + C::OFF_Q + x * C::QTILE + half * C::QHALF + r * 128 +
                                  ((c ^ (r & 7)) << 4)) = v;
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_addr((const void*)(misc + 0))), "r"(C::TMEM_COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];

    auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t role_bit) -> bool {
        if (misc[1]) return false;
        const bool ok = mbar_wait_bounded(smem_addr(bar), parity, p.wait_ns);
        if (!ok) {
            misc[1] = 1u;
            flag_status(p.status, PKV_DEV_TIMEOUT | role_bit);
        }
        return ok;
    };

    if (warp == 0) {
        // ------------------------------------------------------ producer ---
        if (lane == 0) {
            int issued = 0;
            for (int c = 0; c < nch; ++c) {
                const int st = c % kTcStages;
                if (c >= kTcStages && !wait(&kv_empty[st], ((c / kTcStages) - 1) & 1, 0x400u)) break;
                int mask = 0, nl = 0;
                int blk[kTcChunk / kBlockSize];
#pragma unroll
                for (int jj = 0; jj < kTcChunk / kBlockSize; ++jj) {
                    const int j = c * (kTcChunk / kBlockSize) + jj;
                    blk[jj] = -1;
                    if (j <= jmax) {
                        const int x = __ldg(p.block_tables + (long long)b * p.mb + j);
                        if (unsigned(x) < unsigned(p.num_blocks)) {
                            blk[jj] = x;
                            mask |= 1 << jj;
                            ++nl;
                        } else {
                            flag_status(p.status, PKV_DEV_BAD_BLOCK);
                        }
                    }
                }
                smask[st] = mask;
                const uint32_t bar = smem_addr(&kv_full[st]);
                const uint32_t extra = (c == 0 && unit == p.stall_cta) ? 16u : 0u;
                if (nl || extra)
                    mbar_arrive_expect_tx(bar, uint32_t(nl * 2 * C::NH * kBlockSize * 128) + extra);
                else mbar_arrive(bar);
                ++issued;
                unsigned char* sk = smem + C::OFF_KV + st * C::KV_STAGE;
#pragma unroll
                for (int jj = 0; jj < kTcChunk / kBlockSize; ++jj) {
                    if (blk[jj] < 0) continue;
                    const int y = (blk[jj] * p.hkv + kvh) * kBlockSize;
#pragma unroll
                    for (int h = 0; h < C::NH; ++h) {
                        tma_load_2d(smem_addr(sk + h * C::HALF + jj * kBlockSize * 128), &tmk, 64 * h, y, bar);
                        tma_load_2d(smem_addr(sk + (C::NH + h) * C::HALF + jj * kBlockSize * 128), &tmv,
                                    64 * h, y, bar);
                    }
                }
            }
            // After an abort, let the copies of the last chunks issued land
            // (bounded) before the CTA may exit.
            if (misc[1])
                for (int c = max(0, issued - kTcStages); c < issued; ++c)
                    mbar_wait_bounded(smem_addr(&kv_full[c % kTcStages]), (c / kTcStages) & 1,
                                      p.wait_ns);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer ---
        if (lane == 0) {
            const uint32_t ab = std::is_same<KV, BF16>::value ? 1u : 0u;
            const uint32_t id_s = tc_idesc(ab, 0, kTcChunk, kTcRows);
            const uint32_t id_o = tc_idesc(ab, 1, D, kTcRows);
            const uint64_t dq0 = tc_desc(smem_addr(smem + C::OFF_Q), 16, 1024);
            const uint64_t dk0 = tc_desc(smem_addr(smem + C::OFF_KV), 16, 1024);
            const uint64_t dv0 = tc_desc(smem_addr(smem + C::OFF_KV + C::NH * C::HALF), C::HALF, 1024);
            auto issue_s = [&](int c, int x) {
                const uint64_t dq = dq0 + uint64_t((x * C::QTILE) >> 4);
                const uint64_t dk = dk0 + uint64_t((c % kTcStages) * (C::KV_STAGE >> 4));
                const uint32_t d = tmem + x * 2 * kTcChunk + (c & 1) * kTcChunk;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk / 4) * C::QHALF + (kk % 4) * 32) >> 4;
                    const uint32_t offk = ((kk / 4) * C::HALF + (kk % 4) * 32) >> 4;
                    tc_mma(d, dq + off, dk + offk, id_s, kk > 0);
                }
                tc_commit(smem_addr(&s_full[2 * x + (c & 1)]));
            };
            auto issue_pv = [&](int c, int x) {
                const uint64_t dv = dv0 + uint64_t((c % kTcStages) * (C::KV_STAGE >> 4));
                // P of chunk c (hi at columns 0-31, lo at 32-63 of its S buffer)
                const uint32_t tp = tmem + x * 2 * kTcChunk + (c & 1) * kTcChunk;
                const uint32_t to = tmem + 4 * kTcChunk + x * 128;
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int kk = 0; kk < kTcChunk / 16; ++kk)
                        tc_mma_ts(to, tp + part * (kTcChunk / 2) + kk * 8,
                                  dv + uint64_t((kk * 16 * 128) >> 4), id_o,
                                  (c > 0 || part > 0 || kk > 0) ? 1u : 0u);
                tc_commit(smem_addr(&o_done[x]));
            };
            auto finish = [&](int c) -> bool {   // P.V of chunk c for both tiles
                if (!wait(&p_full[0], c & 1, 0x800u)) return false;
                tc_fence_after();
                issue_pv(c, 0);
                if (two) {
                    if (!wait(&p_full[1], c & 1, 0x800u)) return false;
                    tc_fence_after();
                    issue_pv(c, 1);
                }
                tc_commit(smem_addr(&kv_empty[c % kTcStages]));
                return true;
            };
            bool ok = true;
            for (int c = 0; c < nch && ok; ++c) {
                ok = wait(&kv_full[c % kTcStages], (c / kTcStages) & 1, 0x800u);
                if (!ok) break;
                tc_fence_after();
                issue_s(c, 0);
                if (two) issue_s(c, 1);
                if (c > 0) ok = finish(c - 1);
            }
            if (ok) finish(nch - 1);
            tc_commit(smem_addr(&drain[0]));
            mbar_wait_bounded(smem_addr(&drain[0]), 0, 2000000000ull);
        }
    } else {
        // -------------------------------------- softmax + epilogue, per tile ---
        const int x = (warp - 2) >> 2;                        // tile
        if (x == 0 || two) {
            const int r = 32 * (warp & 3) + lane;             // TMEM lane = row of the tile
            const uint32_t lane_addr = uint32_t(32 * (warp & 3)) << 16;
            const uint32_t tm_s = tmem + x * 2 * kTcChunk;
            const uint32_t tm_o = tmem + 4 * kTcChunk + x * 128;
            const int qi = q00 + x * QPT + r / G;
            const bool rv = qi < n;
            const int pos = L - n + qi;
            float m = -INFINITY, l = 0.f;
            const int last_blk_tok = ((L - 1) / kBlockSize) * kBlockSize;
            const bool qpos = p.qscale > 0.f;                  // max of raw scores = max of scaled
            bool ok = true;
            for (int c = 0; c < nch; ++c) {
                const int st = c % kTcStages;
                const int tok0 = c * kTcChunk;
                if (ok) ok = __all_sync(kFull, wait(&s_full[2 * x + (c & 1)], (c >> 1) & 1, 0x1000u));
                if (ok) ok = __all_sync(kFull, wait(&kv_full[st], (c / kTcStages) & 1, 0x1000u));
                float s[kTcChunk];
                float mx = -INFINITY;
                int mask = 0;
                bool plain = false;   // warp-uniform: raw scores, every column visible
                if (ok) {
                    tc_fence_after();
                    tc_ld64(tm_s + lane_addr + (c & 1) * kTcChunk, s);
                    mask = smask[st];
                    plain = __all_sync(kFull, rv && pos - tok0 >= kTcChunk - 1 &&
                                                  mask == (1 << (kTcChunk / kBlockSize)) - 1) && qpos;
                    if (plain) {
                        float mr = s[0];
#pragma unroll
                        for (int i = 1; i < kTcChunk; ++i) mr = fmaxf(mr, s[i]);
                        mx = mr * p.qscale;
                    } else {
#pragma unroll
                        for (int i = 0; i < kTcChunk; ++i) {
                            const int tok = tok0 + i;
                            const bool vis = rv && tok <= pos && ((mask >> (i / kBlockSize)) & 1);
                            s[i] = vis ? s[i] * p.qscale : -INFINITY;
                            mx = fmaxf(mx, s[i]);
                        }
                    }
                }
                if (ok) {
                    const bool grow = mx > m + kTcLazy || (m == -INFINITY && mx > -INFINITY);
                    const bool rescale = c > 0 && __any_sync(kFull, grow && m > -INFINITY);
                    const float a = (grow && m > -INFINITY) ? fast_exp2(m - mx) : 1.f;
                    if (grow && m > -INFINITY) l *= a;
                    if (grow) m = mx;
                    // P = exp2(s - m) as hi + lo 16-bit parts, packed two per
                    // column into this chunk's S buffer (its own TMEM lane), where
                    // the P.V MMAs take it as their A operand
                    const uint32_t tp = tm_s + lane_addr + (c & 1) * kTcChunk;
                    auto emit = [&](auto expo) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t hw[16], lw[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float x0 = expo(s[32 * h + 2 * e]);
                                const float x1 = expo(s[32 * h + 2 * e + 1]);
                                l += x0 + x1;
                                hw[e] = pack2<KV>(x0, x1);
                                const float2 rr = unpack2(KV{}, hw[e]);
                                lw[e] = pack2<KV>(x0 - rr.x, x1 - rr.y);
                            }
                            tc_st16(tp + 16 * h, hw);
                            tc_st16(tp + kTcChunk / 2 + 16 * h, lw);
                        }
                    };
                    if (plain) {   // finite raw scores, m finite: one fma and one ex2 each
                        const float nm = -m, qs = p.qscale;
                        emit([&](float y) { return fast_exp2(fmaf(y, qs, nm)); });
                    } else {
                        emit([&](float y) { return y == -INFINITY ? 0.f : fast_exp2(y - m); });
                    }
                    tc_wait_st();
                    // O may be touched only once the previous chunk's P.V is done
                    if (c > 0) ok = __all_sync(kFull, wait(&o_done[x], (c - 1) & 1, 0x1000u));
                    if (ok && rescale) {
                        tc_fence_after();
#pragma unroll
                        for (int c0 = 0; c0 < D; c0 += 32) {
                            float o[32];
                            tc_ld32(tm_o + lane_addr + c0, o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] *= a;
                            tc_st32(tm_o + lane_addr + c0, o);
                        }
                    }
                    // tile 0 zeroes V rows past the context (both tiles' P.V
                    // follow tile 0's P in the MMA thread's order)
                    if (ok && x == 0 && last_blk_tok >= tok0 && last_blk_tok < tok0 + kTcChunk &&
                        L < last_blk_tok + kBlockSize) {
                        const int jj = (last_blk_tok - tok0) / kBlockSize;
                        if ((mask >> jj) & 1) {
                            const int r0 = L - last_blk_tok;
                            const int nrow = kBlockSize - r0;
                            unsigned char* vb = smem + C::OFF_KV + st * C::KV_STAGE + C::NH * C::HALF;
                            for (int i = r; i < nrow * C::NH * 8; i += kTcRows) {
                                const int row = i / (C::NH * 8), rem = i % (C::NH * 8);
                                const int h = rem / 8, c8 = rem % 8;
                                *reinterpret_cast<uint4*>(vb + h * C::HALF + (jj * kBlockSize + r0 + row) * 128 + c8 * 16) =
                                    make_uint4(0u, 0u, 0u, 0u);
                            }
                        }
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                tc_named_sync(1 + x, kTcRows);
                if (r == 0) mbar_arrive(smem_addr(&p_full[x]));
            }
            if (ok) ok = __all_sync(kFull, wait(&o_done[x], (nch - 1) & 1, 0x1000u));
            if (ok) {
                tc_fence_after();
                const float inv = l > 0.f ? 1.f / l : 0.f;
                uint16_t* dst = static_cast<uint16_t*>(p.out) + ((long long)(cu + qi) * p.hq + kvh * G + r % G) * D;
#pragma unroll
                for (int c0 = 0; c0 < D; c0 += 32) {
                    float o[32];
                    tc_ld32(tm_o + lane_addr + c0, o);
                    if (rv) {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) w[i] = pack2<KV>(o[2 * i] * inv, o[2 * i + 1] * inv);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            reinterpret_cast<uint4*>(dst + c0)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(C::TMEM_COLS));
}

// tcgen05 row-tile path: launchers by cache type, head dim and group size.
template <typename KV, int D, int G>
cudaError_t tc_launch(const CUtensorMap& k, const CUtensorMap& v, const MqParams& p, int grid,
                      cudaStream_t st) {
    // two row tiles per CTA: grid counts tile pairs
    const int smem = TcCfg<D>::BYTES;
    cudaError_t e = cudaFuncSetAttribute(mq_tc_kernel<KV, D, G>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const long long tiles = (long long)grid / p.tmax;
    const int g2 = int(tiles * ((p.tmax + 1) / 2));
    return launch_pdl(mq_tc_kernel<KV, D, G>, dim3(g2), dim3(kTcThreads), size_t(smem), st, k, v, p);
}
template <typename KV, int D>
TcLaunch tc_pick_g(int G) {
    switch (G) {
        case 1: return tc_launch<KV, D, 1>;
        case 2: return tc_launch<KV, D, 2>;
        case 4: return tc_launch<KV, D, 4>;
        case 8: return tc_launch<KV, D, 8>;
    }
    return nullptr;
}
template <typename KV>
TcLaunch tc_pick(int D, int G) {
    if (D == 128) return tc_pick_g<KV, 128>(G);
    if (D == 64) return tc_pick_g<KV, 64>(G);
    return nullptr;
}

}  // namespace
}  // namespace pkv
