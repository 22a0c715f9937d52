// The exact choice of the largest of a row of scores, for one CTA.
//
// Of values [0, n) the first keep_first, the last keep_last and, of the rest,
// the largest are kept, `count` in all (count >= the forced ones, or n), in
// ascending order of index. Equal values go to the lowest index; NaN counts
// as the lowest, -0 as +0.
//
// Floats map to unsigned keys of the same order. One histogram of kBins equal
// intervals over [lowest, highest key] finds the interval of the threshold,
// whatever the values, with few atomics on one address, since the intervals
// follow the row's own range (a fixed radix would put scores of one exponent
// into one or two bins). While the interval holds more than kRanked keys, it
// gets a histogram of its own; the rest are ranked against one another by one
// warp. (Ranking up to 256 keys instead of a second histogram cost 1900
// instructions per warp on 1280 scores, most of them there, and 19 instead of
// 13 us for 512 rows.) Barriers and shared-memory latency bound it, not the
// reads.
#pragma once

#include "common.cuh"

#include <atomic>

namespace pkv {
namespace choose {

constexpr int kBins = 2048;
constexpr int kKeepRow = 32768;  // values of a row kept in shared memory (128 KB), at most

__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);   // -0 -> +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kRanked = 32;      // keys that are ranked against one another, at most

// The value of a key; NaN and zeros lose their sign and payload.
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ bool key_is_lossy(uint32_t k) { return k == 0u || k == 0x80000000u; }

// Shared memory of one CTA of T threads.
template <int T>
struct Scratch {
    union {
        alignas(16) int hist[kBins];
        uint32_t cand[kRanked];
    };
    uint32_t warp_lo[T / 32], warp_hi[T / 32];
    int warp_a[T / 32], warp_b[T / 32];
    uint32_t key;
    int bin, above, in_bin, n_cand;
};

// Kept: key > key_min, or key == key_min among the `ties` lowest indices of it.
struct Threshold {
    uint32_t key_min;
    int ties;
};

// Reads load(i), i in [0, n), puts its keys into `row` (unless nullptr) and notes
// the range of those of [i0, i1). All threads; ends with a barrier.
template <int T, typename Load>
__device__ void take_row(Scratch<T>& s, Load load, uint32_t* row, int n, int i0, int i1) {
    const int t = threadIdx.x;
    uint32_t mn = 0xffffffffu, mx = 0u;
#pragma unroll 4
    for (int i = t; i < n; i += T) {
        const uint32_t k = order_key(load(i));
        if (row) row[i] = k;
        if (i < i0 || i >= i1) continue;
        mn = min(mn, k);
        mx = max(mx, k);
    }
    mn = __reduce_min_sync(kFull, mn);
    mx = __reduce_max_sync(kFull, mx);
    if ((t & 31) == 0) { s.warp_lo[t >> 5] = mn; s.warp_hi[t >> 5] = mx; }
    for (int i = t; i < kBins / 4; i += T) reinterpret_cast<int4*>(s.hist)[i] = make_int4(0, 0, 0, 0);
    if (t == 0) s.n_cand = 0;
    __syncthreads();
}

// The threshold of the `need` largest keys get(i), i in [i0, i1), after take_row.
template <int T, typename Get>
__device__ Threshold find_threshold(Scratch<T>& s, Get get, int i0, int i1, int need) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    if (need <= 0) return Threshold{0xffffffffu, 0};            // no value has this key
    if (need >= i1 - i0) return Threshold{0u, 0x7fffffff};
    uint32_t lo = 0xffffffffu, hi = 0u;
#pragma unroll
    for (int w = 0; w < T / 32; ++w) { lo = min(lo, s.warp_lo[w]); hi = max(hi, s.warp_hi[w]); }
    while (lo < hi) {
        const int bits = 32 - __clz(hi - lo);
        const int shift = bits > 11 ? bits - 11 : 0;
        static_assert(kBins == 1 << 11, "bins of 11 bits");
#pragma unroll 4
        for (int i = i0 + t; i < i1; i += T) {
            const uint32_t k = get(i);
            if (k >= lo && k <= hi) atomicAdd(&s.hist[(k - lo) >> shift], 1);
        }
        __syncthreads();
        // counts from the top: thread t owns bins [b0, b0 + PER)
        constexpr int PER = kBins / T;
        static_assert(PER * T == kBins && PER % 2 == 0, "bins divide over the threads");
        const int b0 = (T - 1 - t) * PER;
        int h[PER], sum = 0;
#pragma unroll
        for (int i = 0; i < PER; i += 2) {
            const int2 v = *reinterpret_cast<const int2*>(&s.hist[b0 + i]);
            h[i] = v.x;
            h[i + 1] = v.y;
            sum += v.x + v.y;
        }
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) s.warp_a[warp] = inc;
        __syncthreads();
        int above = inc - sum;
#pragma unroll
        for (int w = 0; w < T / 32; ++w) above += w < warp ? s.warp_a[w] : 0;
        if (above < need && need <= above + sum) {
#pragma unroll
            for (int i = PER - 1; i >= 0; --i) {
                if (above < need && need <= above + h[i]) { s.bin = b0 + i; s.above = above; s.in_bin = h[i]; }
                above += h[i];
            }
        }
        __syncthreads();
        const int in_bin = s.in_bin;
        need -= s.above;
        const uint32_t base = lo + (uint32_t(s.bin) << shift);
        const uint32_t top = base + ((1u << shift) - 1u);
        hi = top < base || top > hi ? hi : top;
        lo = base;
        if (in_bin == need) return Threshold{lo, 0x7fffffff};   // all of the interval
        if (in_bin <= kRanked) {
#pragma unroll 4
            for (int i = i0 + t; i < i1; i += T) {
                const uint32_t k = get(i);
                if (k >= lo && k <= hi) s.cand[atomicAdd(&s.n_cand, 1)] = k;
            }
            __syncthreads();
            if (t < in_bin) {
                const uint32_t k = s.cand[t];
                int more = 0, same = 0;
                for (int i = 0; i < in_bin; ++i) {
                    const uint32_t x = s.cand[i];
                    more += x > k;
                    same += x == k;
                }
                if (more < need && need <= more + same) { s.key = k; s.above = more; }
            }
            __syncthreads();
            return Threshold{s.key, need - s.above};
        }
        __syncthreads();   // all have read the bins' outcome
        for (int i = t; i < kBins / 4; i += T) reinterpret_cast<int4*>(s.hist)[i] = make_int4(0, 0, 0, 0);
        __syncthreads();
    }
    return Threshold{lo, need};
}

// Calls put(rank, i) for every kept i of a row in shared memory, rank ascending
// with i. Every thread owns a run of the row of odd length (no bank conflicts),
// so that it counts and places its own without a vote per element.
template <int T, typename Put>
__device__ void emit_shared(Scratch<T>& s, const uint32_t* row, int n, int keep_first, int keep_last,
                            Threshold th, Put put) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int per = ((n + T - 1) / T) | 1, lo = min(n, t * per), hi = min(n, lo + per);
    const int last0 = n - keep_last;
    int n_sure = 0, n_tie = 0;
#pragma unroll 4
    for (int i = lo; i < hi; ++i) {
        const uint32_t k = row[i];
        const bool forced = i < keep_first || i >= last0;
        n_sure += forced || k > th.key_min;
        n_tie += !forced && k == th.key_min;
    }
    int sure = n_sure, tie = n_tie;          // inclusive prefixes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(kFull, sure, o), b = __shfl_up_sync(kFull, tie, o);
        if (lane >= o) { sure += a; tie += b; }
    }
    if (lane == 31) { s.warp_a[warp] = sure; s.warp_b[warp] = tie; }
    __syncthreads();
    sure -= n_sure;
    tie -= n_tie;
#pragma unroll
    for (int w = 0; w < T / 32; ++w)
        if (w < warp) { sure += s.warp_a[w]; tie += s.warp_b[w]; }
    int rank = sure + min(tie, th.ties);
#pragma unroll 4
    for (int i = lo; i < hi; ++i) {
        const uint32_t k = row[i];
        bool keep = i < keep_first || i >= last0 || k > th.key_min;
        if (!keep && k == th.key_min) keep = tie++ < th.ties;
        if (keep) put(rank++, i);
    }
}

// The same for a row that is read again: every warp walks one contiguous part.
template <int T, typename Get, typename Put>
__device__ void emit(Scratch<T>& s, Get get, int n, int keep_first, int keep_last, Threshold th,
                     Put put) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = ((n + T - 1) / T) * 32;
    const int lo = min(n, warp * per), hi = min(n, lo + per);
    const int last0 = n - keep_last;
    auto state = [&](int i, bool& sure, bool& tie) {
        sure = tie = false;
        if (i >= hi) return;
        if (i < keep_first || i >= last0) { sure = true; return; }
        const uint32_t k = get(i);
        sure = k > th.key_min;
        tie = k == th.key_min && th.ties > 0;
    };
    int n_sure = 0, n_tie = 0;
    for (int base = lo; base < hi; base += 32) {
        bool sure, tie;
        state(base + lane, sure, tie);
        n_sure += __popc(__ballot_sync(kFull, sure));
        n_tie += __popc(__ballot_sync(kFull, tie));
    }
    if (lane == 0) { s.warp_a[warp] = n_sure; s.warp_b[warp] = n_tie; }
    __syncthreads();
    int rank = 0, tied = 0;
    for (int w = 0; w < warp; ++w) {
        rank += s.warp_a[w] + min(s.warp_b[w], max(0, th.ties - tied));
        tied += s.warp_b[w];
    }
    const unsigned below = (1u << lane) - 1u;
    for (int base = lo; base < hi; base += 32) {
        bool sure, tie;
        state(base + lane, sure, tie);
        const unsigned m_tie = __ballot_sync(kFull, tie);
        const bool keep = sure || (tie && tied + __popc(m_tie & below) < th.ties);
        const unsigned m_keep = __ballot_sync(kFull, keep);
        if (keep) put(rank + __popc(m_keep & below), base + lane);
        rank += __popc(m_keep);
        tied += __popc(m_tie);
    }
}

// Keeps `count` of load(0 .. n-1) (see the file comment), n > count: put(rank, i,
// key). `row` keeps the keys between the passes, or nullptr. All threads.
template <int T, typename Load, typename Put>
__device__ void choose_row(Scratch<T>& s, Load load, uint32_t* row, int n, int keep_first,
                           int keep_last, int count, Put put) {
    const int need = count - keep_first - keep_last;
    take_row(s, load, row, n, keep_first, n - keep_last);
    if (row) {
        const Threshold th = find_threshold(s, [&](int i) { return row[i]; }, keep_first, n - keep_last, need);
        emit_shared(s, row, n, keep_first, keep_last, th, [&](int rank, int i) { put(rank, i, row[i]); });
    } else {
        auto key = [&](int i) { return order_key(load(i)); };
        const Threshold th = find_threshold(s, key, keep_first, n - keep_last, need);
        emit(s, key, n, keep_first, keep_last, th, [&](int rank, int i) { put(rank, i, key(i)); });
    }
}

// Threads per row of a call whose rows hold up to `width` values. Latency bounds a
// row, so more threads shorten long rows, until rows share SMs; rows that fill
// shared memory share none. Microseconds with 256 / 512 / 1024 threads, all rows
// full, a 16th of them (at least 32) chosen:
//   width     64 rows             304                 608                 1024
//    1024  4.2  4.4  6.5    4.8  7.3 12.4    8.1 10.8 23.7   10.4 15.8 39.7
//    4096  7.7  6.6  8.4    8.5 11.1 15.6   15.1 16.7 30.4   18.9 24.6 51.1
//    8192 11.4  9.0 10.1   13.1 15.5 19.6   21.3 21.7 36.7   29.8 34.5 62.2
//   16384 19.4 13.8 13.4   25.0 18.8 26.0   41.2 34.3 49.5   63.3 55.4 84.0
//   32768 35.3 23.1 20.0   69.5 45.4 39.2    151 97.1 79.5    292  188  148
// At 152 rows (one per SM) 256 and 512 are even at a width of 2048 (5.6); at 153 to
// 304 rows 256 is ahead or even up to 4096 and up to 1.2 us behind at 8192.
// Eviction, whose 64 kept rows of each move too, shows the same order (8192 tokens:
// 13.2 10.9 11.5, 15.3 14.3 21.6, 25.3 24.6 38.9, 36.1 38.9 62.9).
inline int threads_per_row(long long width, long long rows) {
    if (width > 16384) return 1024;
    return width > 8192 || (rows <= 152 && width > 2048) ? 512 : 256;
}

// Launches one CTA of T threads per row, with room for p.cap values of it. Beyond
// 48 KB a kernel needs leave for its shared memory, and the leave belongs to the
// kernel, not to the call: asking for what this call needs would lower it under a
// launch of another host thread. So the most is asked for, whatever the row, once
// per device and again where a launch fails (a further context, a reset device).
template <auto Kernel, int T, typename P>
cudaError_t launch_rows(const P& p, int rows, cudaStream_t st) {
    static std::atomic<unsigned long long> leave{0};
    const size_t smem = size_t(p.cap) * sizeof(uint32_t);
    if (smem + sizeof(Scratch<T>) <= 48 * 1024)
        return launch_pdl(Kernel, dim3(rows), dim3(T), smem, st, p);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (leave.load(std::memory_order_relaxed) & bit) {
        if (launch_pdl(Kernel, dim3(rows), dim3(T), smem, st, p) == cudaSuccess) return cudaSuccess;
        cudaGetLastError();
    }
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kKeepRow * int(sizeof(uint32_t)));
    if (e == cudaSuccess) e = launch_pdl(Kernel, dim3(rows), dim3(T), smem, st, p);
    if (e == cudaSuccess) leave.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

}  // namespace choose
}  // namespace pkv
