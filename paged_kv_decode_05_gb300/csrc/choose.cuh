// The exact choice of the largest of a row of scores, for one CTA.
//
// Of values [0, n) the first keep_first, the last keep_last and, of the rest,
// the largest are kept, `count` in all (count >= the forced ones, or n), in
// ascending order of index. Equal values go to the lowest index; NaN counts
// as the lowest, -0 as +0.
//
// Floats map to unsigned keys of the same order. The threshold is found by
// histograms of kBins equal intervals over [lowest, highest key still in
// question], which narrow it by a factor of kBins each time: two or three
// reads of the row whatever the values, and few atomics on one address, since
// the intervals follow the row's own range (a fixed radix would put scores of
// one exponent into one or two bins).
#pragma once

#include "common.cuh"

namespace pkv {
namespace choose {

constexpr int kBins = 2048;

__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);   // -0 -> +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Shared memory of one CTA of T threads.
template <int T>
struct Scratch {
    int hist[kBins];
    int warp_a[T / 32], warp_b[T / 32];
    uint32_t lo, hi;
    int bin, above, in_bin;
};

// Kept: key > key_min, or key == key_min among the `ties` lowest indices of it.
struct Threshold {
    uint32_t key_min;
    int ties;
};

// The threshold of the `need` largest of get(i), i in [i0, i1). All threads.
template <int T, typename Get>
__device__ Threshold find_threshold(Scratch<T>& s, Get get, int i0, int i1, int need) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    if (need <= 0) return Threshold{0xffffffffu, 0};            // no value has this key
    if (need >= i1 - i0) return Threshold{0u, 0x7fffffff};
    // range of the keys
    uint32_t mn = 0xffffffffu, mx = 0u;
    for (int i = i0 + t; i < i1; i += T) {
        const uint32_t k = order_key(get(i));
        mn = min(mn, k);
        mx = max(mx, k);
    }
    mn = __reduce_min_sync(kFull, mn);
    mx = __reduce_max_sync(kFull, mx);
    if (t == 0) { s.lo = 0xffffffffu; s.hi = 0u; }
    __syncthreads();
    if (lane == 0) { atomicMin(&s.lo, mn); atomicMax(&s.hi, mx); }
    __syncthreads();
    uint32_t lo = s.lo, hi = s.hi;
    while (lo < hi) {
        const int bits = 32 - __clz(hi - lo);
        const int shift = bits > 11 ? bits - 11 : 0;
        static_assert(kBins == 1 << 11, "bins of 11 bits");
        for (int i = t; i < kBins; i += T) s.hist[i] = 0;
        __syncthreads();
        for (int i = i0 + t; i < i1; i += T) {
            const uint32_t k = order_key(get(i));
            if (k >= lo && k <= hi) atomicAdd(&s.hist[(k - lo) >> shift], 1);
        }
        __syncthreads();
        // counts from the top: thread t owns bins [b0, b0 + PER)
        constexpr int PER = kBins / T;
        static_assert(PER * T == kBins && PER >= 1, "bins divide over the threads");
        const int b0 = (T - 1 - t) * PER;
        int sum = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) sum += s.hist[b0 + i];
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) s.warp_a[warp] = inc;
        __syncthreads();
        int above = inc - sum;
        for (int w = 0; w < warp; ++w) above += s.warp_a[w];
        if (above < need && need <= above + sum) {
            int b = b0 + PER - 1;
            while (above + s.hist[b] < need) above += s.hist[b--];
            s.bin = b;
            s.above = above;
            s.in_bin = s.hist[b];
        }
        __syncthreads();
        need -= s.above;
        const uint32_t base = lo + (uint32_t(s.bin) << shift);
        const uint32_t top = base + ((1u << shift) - 1u);
        hi = top < base || top > hi ? hi : top;
        lo = base;
        const bool all = s.in_bin == need;
        __syncthreads();   // the next turn overwrites what was read here
        if (all) return Threshold{lo, 0x7fffffff};
    }
    return Threshold{lo, need};
}

// Calls put(rank, i) for every kept i of [0, n), rank ascending with i. All
// threads; every warp walks one contiguous part of the row.
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
        const uint32_t k = order_key(get(i));
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

// Keeps `count` of get(0 .. n-1) (see the file comment). All threads.
template <int T, typename Get, typename Put>
__device__ void choose_row(Scratch<T>& s, Get get, int n, int keep_first, int keep_last, int count,
                           Put put) {
    keep_first = min(keep_first, n);
    keep_last = min(keep_last, n - keep_first);
    const int need = count - keep_first - keep_last;
    const Threshold th = find_threshold(s, get, keep_first, n - keep_last, need);
    emit(s, get, n, keep_first, keep_last, th, put);
}

}  // namespace choose
}  // namespace pkv
