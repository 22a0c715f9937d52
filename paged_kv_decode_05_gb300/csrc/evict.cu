// Eviction from the cache by accumulated attention weight.
//
// Every (sequence, kv head) keeps its first and last tokens and, of the rest,
// the ones with the largest accumulated weight, `budget` in all. Two kernels:
//   choose  one CTA per (sequence, kv head): the exact choice (choose.cuh),
//           the kept positions in order and their weights;
//   move    the kept rows of K and V become rows 0, 1, 2, ... of the new
//           block table; for INT8, a new tile's scale is the largest of its
//           rows' old scales and codes become rne(code * s_old / s_new).
// Bound by memory: 4 bytes per token, and 2 D elements read and written per
// kept token and kv head. 48 sequences of 2k to 12k tokens cut to 2048, 8 heads
// of 128 in 16 bits: 145 us, of which the move of 805 MB takes 122 (0.98 of the
// measured copy rate) and the choice, bound by latency, the rest.
//
// In place (the new table names old blocks at their own places) the move is safe
// because the kept positions ascend: row r comes from a position >= r, so every
// source of a later tile lies at or behind that tile. One CTA then walks a
// (sequence, kv head) in order, loading a group of tiles before it stores any of
// it. Otherwise the tiles of a (sequence, kv head) are shared by several CTAs.
// Which it is, is read from the tables: they may be copies of one another. (The
// cut above in place: 207 us; two sequences to 1000 tokens 8.7 us, in place 42.)
#include "choose.cuh"

namespace pkv {
namespace {

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

struct EvictParams {
    unsigned char* k_cache;
    unsigned char* v_cache;
    float* k_scales;
    float* v_scales;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const float* mass;           // [batch, hkv, mb * 16]
    const int32_t* new_tables;   // [batch, new_mb]
    int32_t* new_lens;           // [batch]
    float* new_mass;             // [batch, hkv, new_mb * 16]
    int32_t* kept;               // [batch, hkv, budget]
    uint32_t* status;
    int hkv, mb, new_mb, num_blocks, budget, keep_first, keep_last;
    int cap;                     // choose: weights that the shared row holds
    int splits;                  // move: CTAs per (sequence, kv head), of which the first
                                 // has all groups where the sequence is compacted in place
};

// Length of sequence b; a length that does not fit its table keeps nothing.
__device__ __forceinline__ int evict_len(const EvictParams& p, int b, bool flag) {
    const int L = p.context_lens[b];
    if (L >= 0 && L <= (long long)p.mb * kBlockSize) return L;
    if (flag) flag_status(p.status, PKV_DEV_BAD_LENGTH);
    return 0;
}

// At least 1536 resident threads per SM (42 registers each): 384 rows then run in
// one wave of CTAs of 512.
template <int T>
__global__ void __launch_bounds__(T, 1536 / T) evict_choose_kernel(const EvictParams p) {
    extern __shared__ uint32_t row[];
    __shared__ choose::Scratch<T> s;
    griddep_wait();
    griddep_launch_dependents();
    const int seg = blockIdx.x, b = seg / p.hkv, kvh = seg - b * p.hkv, t = threadIdx.x;
    const int n = evict_len(p, b, kvh == 0 && t == 0), count = min(n, p.budget);
    const float* src = p.mass + (long long)seg * p.mb * kBlockSize;
    int32_t* kept = p.kept + (long long)seg * p.budget;
    float* nm = p.new_mass + (long long)seg * p.new_mb * kBlockSize;
    if (kvh == 0 && t == 0) p.new_lens[b] = count;
    for (int i = count + t; i < p.budget; i += T) kept[i] = -1;
    for (int i = count + t; i < p.new_mb * kBlockSize; i += T) nm[i] = 0.f;
    if (count == n) {
        for (int i = t; i < n; i += T) {
            kept[i] = i;
            nm[i] = __ldcg(src + i);
        }
        return;
    }
    choose::choose_row<T>(s, [&](int i) { return __ldcg(src + i); }, n <= p.cap ? row : nullptr, n,
                          p.keep_first, p.keep_last, count, [&](int rank, int i, uint32_t key) {
                              kept[rank] = i;
                              nm[rank] = choose::key_is_lossy(key) ? __ldcg(src + i)
                                                                   : choose::key_value(key);
                          });
}

constexpr int kMoveThreads = 256;

// Tiles (16 rows of K and V) moved together: enough for two 16-byte vectors of
// each of K and V per thread.
template <int ROW> struct MoveCfg {
    static constexpr int VPR = ROW / 16;                     // vectors per row
    static constexpr int VPT = kBlockSize * VPR;             // vectors per tile
    static constexpr int TILES = 2 * kMoveThreads / VPT;     // tiles per group
    static constexpr int ROWS = TILES * kBlockSize;
    static_assert(TILES >= 1 && ROWS <= kMoveThreads, "one thread looks up each row");
};

template <bool I, int ROW>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
    using C = MoveCfg<ROW>;
    __shared__ long long s_src[C::ROWS];     // source row (units of rows), -1: none
    __shared__ long long s_dst[C::TILES];    // destination tile, -1: none
    __shared__ float s_scale[C::ROWS][2];    // INT8: the source rows' scales
    __shared__ int s_move[C::TILES];         // some row of the tile changes its place
    griddep_wait();
    griddep_launch_dependents();
    const int t = threadIdx.x;
    const int seg = blockIdx.x / p.splits, part = blockIdx.x - seg * p.splits;
    const int b = seg / p.hkv, kvh = seg - b * p.hkv;
    const int count = min(evict_len(p, b, false), p.budget);
    const int tiles = (count + kBlockSize - 1) / kBlockSize;
    const int groups = (tiles + C::TILES - 1) / C::TILES;
    const int32_t* kept = p.kept + (long long)seg * p.budget;
    int step = p.splits;
    bool ask = step > 1;        // whether the sequence is compacted in place is open
    for (int g = part; g < groups; g += step) {
        const int tile0 = g * C::TILES, r0 = tile0 * kBlockSize + t;
        const int at = t < C::ROWS && r0 < count ? __ldcg(kept + r0) : 0;
        if (t < C::TILES) {
            long long dst = -1;
            if (tile0 + t < tiles) {
                const int blk = p.new_tables[(long long)b * p.new_mb + tile0 + t];
                if (unsigned(blk) < unsigned(p.num_blocks)) dst = (long long)blk * p.hkv + kvh;
                else if (kvh == 0) flag_status(p.status, PKV_DEV_BAD_BLOCK);
            }
            s_dst[t] = dst;
            s_move[t] = 0;
        }
        if (ask) {
            ask = false;
            bool same = false;      // by the warps that look nothing else up
            for (int i = t - 32; i >= 0 && i < tiles; i += kMoveThreads - 32)
                same = same || p.new_tables[(long long)b * p.new_mb + i] == p.block_tables[(long long)b * p.mb + i];
            if (__syncthreads_or(same)) {
                if (part != 0) return;
                step = 1;
            }
        } else {
            __syncthreads();
        }
        if (t < C::ROWS) {
            long long src = -1;
            if (r0 < count) {
                const int blk = p.block_tables[(long long)b * p.mb + at / kBlockSize];
                const long long dst = s_dst[t / kBlockSize];
                if (unsigned(blk) < unsigned(p.num_blocks)) {
                    const long long tile = (long long)blk * p.hkv + kvh;
                    src = tile * kBlockSize + at % kBlockSize;
                    if constexpr (I) {
                        s_scale[t][0] = p.k_scales[tile];
                        s_scale[t][1] = p.v_scales[tile];
                    }
                } else {
                    flag_status(p.status, PKV_DEV_BAD_BLOCK);
                    if constexpr (I) s_scale[t][0] = s_scale[t][1] = 0.f;
                }
                if (dst >= 0 && src != dst * kBlockSize + r0 % kBlockSize) s_move[t / kBlockSize] = 1;
            } else if constexpr (I) {
                s_scale[t][0] = s_scale[t][1] = 0.f;
            }
            s_src[t] = src;
        }
        __syncthreads();
        // two vectors of K and of V per thread, all loaded before any is stored
        uint4 kx[2], vx[2];
        bool live[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int x = t + i * kMoveThreads, r = x / C::VPR, c = x % C::VPR, tile = r / kBlockSize;
            kx[i] = vx[i] = make_uint4(0u, 0u, 0u, 0u);
            live[i] = s_dst[tile] >= 0 && s_move[tile] && tile0 * kBlockSize + r < count;
            if (live[i] && s_src[r] >= 0) {
                const long long off = s_src[r] * ROW + c * 16;
                kx[i] = __ldcg(reinterpret_cast<const uint4*>(p.k_cache + off));
                vx[i] = __ldcg(reinterpret_cast<const uint4*>(p.v_cache + off));
            }
        }
        float sk[2], sv[2];
        if constexpr (I) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int x = t + i * kMoveThreads, r = x / C::VPR, tile = r / kBlockSize;
                float a = 0.f, c = 0.f;
#pragma unroll
                for (int k = 0; k < kBlockSize; ++k) {
                    a = fmaxf(a, s_scale[tile * kBlockSize + k][0]);
                    c = fmaxf(c, s_scale[tile * kBlockSize + k][1]);
                }
                sk[i] = a;
                sv[i] = c;
                auto grow = [](uint4& v, float s_o, float s) {
                    if (s_o == s || s == 0.f) return;
                    v = make_uint4(requant_word(v.x, s_o, s), requant_word(v.y, s_o, s),
                                   requant_word(v.z, s_o, s), requant_word(v.w, s_o, s));
                };
                grow(kx[i], s_scale[r][0], a);
                grow(vx[i], s_scale[r][1], c);
            }
        }
        __syncthreads();   // every load of the group is done, the lookups may be overwritten
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (!live[i]) continue;
            const int x = t + i * kMoveThreads, r = x / C::VPR, c = x % C::VPR, tile = r / kBlockSize;
            const long long off = (s_dst[tile] * kBlockSize + r % kBlockSize) * ROW + c * 16;
            *reinterpret_cast<uint4*>(p.k_cache + off) = kx[i];
            *reinterpret_cast<uint4*>(p.v_cache + off) = vx[i];
            if constexpr (I) {
                if (r % kBlockSize == 0 && c == 0) {
                    p.k_scales[s_dst[tile]] = sk[i];
                    p.v_scales[s_dst[tile]] = sv[i];
                }
            }
        }
        __syncthreads();
    }
}

template <int T>
cudaError_t launch_choose(const EvictParams& p, int rows, cudaStream_t st) {
    return choose::launch_rows<evict_choose_kernel<T>, T>(p, rows, st);
}

template <bool I, int ROW>
cudaError_t launch_move(EvictParams p, int rows, bool in_place, cudaStream_t st) {
    const int groups = (p.budget + MoveCfg<ROW>::ROWS - 1) / MoveCfg<ROW>::ROWS;
    p.splits = in_place ? 1 : groups;
    if ((long long)rows * p.splits > 0x7fffffffLL) p.splits = 1;
    return launch_pdl(evict_move_kernel<I, ROW>, dim3(unsigned(rows) * unsigned(p.splits)),
                      dim3(kMoveThreads), 0, st, p);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_evict_tokens(void* k_cache, void* v_cache, float* k_scales,
                                       float* v_scales, const pkv_cache_desc* cache,
                                       const int32_t* block_tables, int32_t max_blocks_per_seq,
                                       const int32_t* context_lens, const float* mass,
                                       int32_t batch, int32_t budget, int32_t keep_first,
                                       int32_t keep_last, const int32_t* new_tables,
                                       int32_t new_max_blocks, int32_t* new_lens, float* new_mass,
                                       int32_t* kept, uint32_t* dev_status, cudaStream_t stream) {
    if (!cache || cache->num_blocks <= 0 || cache->num_kv_heads <= 0 || cache->head_dim <= 0)
        return PKV_ERR_INVALID_ARG;
    if (cache->kv_dtype != PKV_F16 && cache->kv_dtype != PKV_BF16 && cache->kv_dtype != PKV_I8)
        return PKV_ERR_INVALID_ARG;
    if (cache->block_size != kBlockSize || (cache->head_dim != 64 && cache->head_dim != 128))
        return PKV_ERR_UNSUPPORTED;
    constexpr int kMaxBlocks = 0x7fffffff / kBlockSize;
    if (batch < 0 || max_blocks_per_seq <= 0 || max_blocks_per_seq > kMaxBlocks || budget <= 0 ||
        keep_first < 0 || keep_last < 0 || (long long)keep_first + keep_last > budget ||
        new_max_blocks <= 0 || new_max_blocks > kMaxBlocks || budget > new_max_blocks * kBlockSize)
        return PKV_ERR_INVALID_ARG;
    if (batch == 0) return PKV_OK;
    if (!k_cache || !v_cache || !block_tables || !context_lens || !mass || !new_tables ||
        !new_lens || !new_mass || !kept)
        return PKV_ERR_INVALID_ARG;
    if (!aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || !aligned_to(block_tables, 4) ||
        !aligned_to(context_lens, 4) || !aligned_to(mass, 4) || !aligned_to(new_tables, 4) ||
        !aligned_to(new_lens, 4) || !aligned_to(new_mass, 4) || !aligned_to(kept, 4) ||
        !aligned_to(dev_status, 4))
        return PKV_ERR_INVALID_ARG;
    const bool i8 = cache->kv_dtype == PKV_I8;
    if (i8 && (!k_scales || !v_scales || !aligned_to(k_scales, 4) || !aligned_to(v_scales, 4)))
        return PKV_ERR_INVALID_ARG;
    const bool in_place = new_tables == block_tables;
    if (in_place && new_max_blocks != max_blocks_per_seq) return PKV_ERR_INVALID_ARG;
    const long long rows = (long long)batch * cache->num_kv_heads;
    if (rows > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
    // read by some CTAs while others write their share
    const size_t lens_bytes = size_t(batch) * 4, row_bytes = size_t(rows) * kBlockSize * 4;
    if (overlap(new_lens, lens_bytes, context_lens, lens_bytes) ||
        overlap(new_mass, row_bytes * new_max_blocks, mass, row_bytes * max_blocks_per_seq))
        return PKV_ERR_INVALID_ARG;
    EvictParams p;
    p.k_cache = static_cast<unsigned char*>(k_cache);
    p.v_cache = static_cast<unsigned char*>(v_cache);
    p.k_scales = k_scales; p.v_scales = v_scales;
    p.block_tables = block_tables; p.context_lens = context_lens; p.mass = mass;
    p.new_tables = new_tables; p.new_lens = new_lens; p.new_mass = new_mass; p.kept = kept;
    p.status = dev_status;
    p.hkv = cache->num_kv_heads; p.mb = max_blocks_per_seq; p.new_mb = new_max_blocks;
    p.num_blocks = cache->num_blocks;
    p.budget = budget; p.keep_first = keep_first; p.keep_last = keep_last;
    const long long width = (long long)max_blocks_per_seq * kBlockSize;
    p.cap = int(width < choose::kKeepRow ? width : choose::kKeepRow);
    p.splits = 1;
    const int threads = choose::threads_per_row(width, rows);
    cudaError_t e = threads == 1024  ? launch_choose<1024>(p, int(rows), stream)
                    : threads == 512 ? launch_choose<512>(p, int(rows), stream)
                                     : launch_choose<256>(p, int(rows), stream);
    if (e != cudaSuccess) return PKV_ERR_CUDA;
    const int D = cache->head_dim;
    if (i8)
        e = D == 128 ? launch_move<true, 128>(p, int(rows), in_place, stream)
                     : launch_move<true, 64>(p, int(rows), in_place, stream);
    else
        e = D == 128 ? launch_move<false, 256>(p, int(rows), in_place, stream)
                     : launch_move<false, 128>(p, int(rows), in_place, stream);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
