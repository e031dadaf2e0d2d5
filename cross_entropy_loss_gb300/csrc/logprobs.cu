// Log probability of a given token, entropy and the K most likely tokens of every row
// of logits -- what a server answering with log probabilities, a policy-gradient step
// or a teacher writing down its distribution takes from the LM head.  With z = x / T:
//
//   m = max_j x_j     S = sum_j e^{(x_j - m) / T}     A = sum_j e^{(x_j - m) / T} (x_j - m) / T
//   lse = m / T + ln S     logp_j = (x_j - m) / T - ln S     H = ln S - A / S
//
// One read of the row gives m, S and A (running sums per thread, rescaled at a new
// maximum).  The top K come out of the same read: a thread's 64-byte block of a chunk
// has one maximum, which the sums need anyway and which is kept as an ordered integer
// key.  Blocks are contiguous, so the K largest blocks by (maximum, lower index first)
// hold the K largest elements by (value, lower index first): with a total order an
// element outside those blocks has K larger ones before it.  So a row's end is
//
//   1. a threshold on the block maxima with at least K and at most 256 blocks at or
//      above it (bisection on the keys, a count over the CTA each step; ties beyond 256
//      blocks are cut by a second bisection on the block index);
//   2. one block a thread, re-read (from L2: the row just went through), and its elements
//      at or above the threshold put on a list;
//   3. each listed element's rank = the number of larger ones, its place in the output.
//
// Rows go to CTAs round-robin; when there are fewer rows than SMs a cluster shares each
// row, joins its sums and lists through distributed shared memory, and ranks every
// CTA's K candidates against the others'.
#include <algorithm>
#include <map>
#include <mutex>

#include "row_stream.cuh"

namespace foak {

namespace {

constexpr int kListCap = 1024;  // listed elements of a row (or of a CTA's share of it)
constexpr int kSelCap = 256;    // blocks they are taken from

struct LogprobParams {
    StreamSrc src;
    float inv_t;       // 1 / T
    ExpScale scale;
    int top_k;
    float* logp;       // [N] or null
    float* entropy;    // [N] or null
    float* lse;        // [N] or null
    float2* stats;     // [N] or null: (m, ln S)
    float* top_lp;     // [N][top_k]
    int32_t* top_ids;  // [N][top_k]
    int32_t* err;
    CeWsHeader* ws;
};

// Unsigned integers in the order of the floats; -0 and +0 are the same key, 0 is no float's key.
__device__ __forceinline__ uint32_t key_of(float f) {
    const uint32_t b = __float_as_uint(f == 0.f ? 0.f : f);
    return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float float_of_key(uint32_t k) {
    return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xffffffffu));
}
// Block maxima are kept as the key's upper half for bf16 (whose lower half is constant) and whole for fp32.
template <int ES>
struct BlockKey {
    using type = uint32_t;
    static __device__ __forceinline__ uint32_t of(float f) { return key_of(f); }
    static __device__ __forceinline__ uint32_t element(uint32_t k) { return k; }  // no element of it has a smaller key
    static __device__ __forceinline__ float value(uint32_t k) { return float_of_key(k); }
};
template <>
struct BlockKey<2> {
    using type = uint16_t;
    static __device__ __forceinline__ uint32_t of(float f) { return key_of(f) >> 16; }
    static __device__ __forceinline__ uint32_t element(uint32_t k) { return k << 16; }
    static __device__ __forceinline__ float value(uint32_t k) {  // the lower half of a negative number's key is ones
        return float_of_key(k >> 15 ? k << 16 : k << 16 | 0xffffu);
    }
};

struct TopScratch {
    int count[2][kStreamWarps];                // partial counts, by the parity of the count
    int n_sel, n_list, n_tied;
    uint32_t thread_max[kStreamThreads];       // key of the largest of a thread's blocks; 0: it has none
    int sel[kSelCap];                          // the chosen blocks
    alignas(16) unsigned long long list[kListCap];  // (key << 32) | ~column
    unsigned long long best[kStreamThreads];   // this CTA's top K in order (clusters)
};

// The sum of n over the consumer threads; one consumer barrier.
__device__ __forceinline__ int consumers_count(int n, TopScratch& t, uint32_t& turn) {
    n = __reduce_add_sync(0xffffffffu, n);
    const uint32_t b = turn++ & 1u;
    if ((threadIdx.x & 31) == 0) t.count[b][threadIdx.x >> 5] = n;
    consumers_sync();
    int s = 0;
#pragma unroll
    for (int w = 0; w < kStreamWarps; ++w) s += t.count[b][w];
    return s;
}

// Places for n entries of each lane in a list whose length is *len: one atomic a warp.
// Returns the lane's first place.
__device__ __forceinline__ int warp_places(int n, int* len) {
    const int lane = threadIdx.x & 31;
    int sum = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += o;
    }
    int base = 0;
    if (lane == 31 && sum) base = atomicAdd(len, sum);
    return __shfl_sync(0xffffffffu, base, 31) + sum - n;
}

// Block `id` of the slice: 0 the head scalars, 1 .. nblk the body's blocks, nblk + 1 the tail scalars.
template <int ES>
struct BlockElements {
    static constexpr int EPV = 16 / ES;
    static constexpr int N = kBlockVec * EPV;
    uint32_t w[kBlockVec * 4];  // the elements as they lie in memory
    int n;
    int64_t col;

    __device__ __forceinline__ void load(const Slice& s, int id, int nblk) {
#pragma unroll
        for (int i = 0; i < kBlockVec * 4; ++i) w[i] = 0;
        if (id > 0 && id <= nblk) {
            const int v0 = (id - 1) * kBlockVec;
            const int nv = min(kBlockVec, s.nv - v0);
            col = s.col0 + static_cast<int64_t>(v0) * EPV;
            n = nv * EPV;
            const uint4* v = reinterpret_cast<const uint4*>(s.body) + v0;
#pragma unroll
            for (int i = 0; i < kBlockVec; ++i) {
                if (i < nv) {
                    const uint4 q = ld_global_v4(v + i);
                    w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
                }
            }
            return;
        }
        col = id ? s.tail_col : 0;
        n = id ? s.t : s.h;
#pragma unroll
        for (int e = 0; e < kMaxScalars; ++e) {
            if (e >= n) continue;
            if constexpr (ES == 2)
                w[e / 2] |= static_cast<uint32_t>(*reinterpret_cast<const unsigned short*>(s.rowp + (col + e) * 2)) << (e & 1) * 16;
            else w[e] = *reinterpret_cast<const uint32_t*>(s.rowp + (col + e) * 4);
        }
    }
    // element e as (key << 32) | ~column, 0 where there is none
    __device__ __forceinline__ unsigned long long item(int e) const {
        float f;
        if constexpr (ES == 2) f = e & 1 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
        else f = __uint_as_float(w[e]);
        return e < n ? (static_cast<unsigned long long>(key_of(f)) << 32) | static_cast<uint32_t>(~static_cast<uint32_t>(col + e))
                     : 0ull;
    }
};

// The slow way to the list, for rows in which the fast one meets more blocks or elements
// than it has room for (many equal values, or a share of few blocks): exact bisections,
// first for the K-th largest block by (maximum, lower index first), then, if need be, for
// the K-th largest element.  nreal > K blocks, or all of them are taken.
template <int ES>
__device__ __noinline__ void top_list_exact(const Slice s, const typename BlockKey<ES>::type* keys, int K, TopScratch& t) {
    using BK = BlockKey<ES>;
    const int tid = threadIdx.x;
    const int nblk = (s.nv + kBlockVec - 1) / kBlockVec;
    const int nreal = nblk + (s.h > 0) + (s.t > 0);
    uint32_t turn = 0;
    consumers_sync();
    if (tid == 0) {
        t.n_sel = 0;
        t.n_list = 0;
    }
    // ---- the blocks: keys above lo, and of those equal to lo the ids up to last
    uint32_t lo = 1;
    int last = 0x7fffffff;
    if (nreal > K) {
        uint32_t hi = ES == 2 ? 0x10000u : 0xffffffffu;  // no key is as large (a NaN's would be)
        int c_lo = nreal, c_hi = 0;                      // blocks at or above lo and hi
        while (hi - lo > 1 && c_lo > kSelCap) {
            const uint32_t mid = lo + (hi - lo) / 2;
            int n = 0;
            for (int b = tid; b < nblk + 2; b += kStreamThreads) n += keys[b] >= mid;
            n = consumers_count(n, t, turn);
            if (n >= K) {
                lo = mid;
                c_lo = n;
            } else {
                hi = mid;
                c_hi = n;
            }
        }
        if (c_lo > kSelCap) {  // hi == lo + 1: ties at lo, the first `need` of them
            const int need = K - c_hi;
            int j0 = -1, j1 = nblk + 1;  // fewer than need ties up to j0, enough up to j1
            while (j1 - j0 > 1) {
                const int mid = j0 + (j1 - j0) / 2;
                int n = 0;
                for (int b = tid; b <= mid; b += kStreamThreads) n += keys[b] == lo;
                if (consumers_count(n, t, turn) >= need) j1 = mid;
                else j0 = mid;
            }
            last = j1;
        }
    }
    consumers_sync();
    for (int b = tid; b < nblk + 2; b += kStreamThreads) {
        const uint32_t k = keys[b];
        if (k > lo || (k == lo && b <= last)) {
            const int i = atomicAdd(&t.n_sel, 1);
            if (i < kSelCap) t.sel[i] = b;
        }
    }
    consumers_sync();
    // ---- one block a thread, and its elements
    const int n_sel = min(t.n_sel, kSelCap);
    BlockElements<ES> el;
    el.n = 0;
    el.col = 0;
    if (tid < n_sel) el.load(s, t.sel[tid], nblk);
    auto at_least = [&](unsigned long long f) {
        int n = 0;
#pragma unroll
        for (int e = 0; e < BlockElements<ES>::N; ++e) n += el.item(e) >= f;
        return consumers_count(n, t, turn);
    };
    // every count is at least K at b0 (or takes every element) and less than K at b1
    unsigned long long b0 = static_cast<unsigned long long>(BK::element(lo)) << 32, b1 = ~0ull;
    if (at_least(b0) > kListCap) {
        while (b1 - b0 > 1) {
            const unsigned long long mid = b0 + (b1 - b0) / 2;
            const int c = at_least(mid);
            if (c >= K) {
                b0 = mid;
                if (c <= kListCap) break;
            } else {
                b1 = mid;
            }
        }
    }
#pragma unroll
    for (int e = 0; e < BlockElements<ES>::N; ++e) {
        const unsigned long long it = el.item(e);
        if (it >= b0) {
            const int i = atomicAdd(&t.n_list, 1);
            if (i < kListCap) t.list[i] = it;
        }
    }
    consumers_sync();
}

// This CTA's largest elements of its slice onto t.list: at least the min(K, all) largest
// ones, at most kListCap.  Returns how many.  keys[1 .. nblk] are the block maxima, keys[0]
// and keys[nblk + 1] those of the head and tail (0: none), t.thread_max the threads'; all
// of them written before a barrier.
template <int ES>
__device__ __forceinline__ int top_list(const Slice& s, const typename BlockKey<ES>::type* keys, int K, TopScratch& t) {
    using BK = BlockKey<ES>;
    constexpr int EPV = 16 / ES;
    constexpr int PER = kStreamThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31;
    const int nblk = (s.nv + kBlockVec - 1) / kBlockVec;
    // A threshold that K threads' maxima, so K blocks, reach: the K-th largest of the 256
    // thread maxima, or a little below it.  Every warp finds it for itself, without a
    // barrier.  Of blocks in random order about -256 ln(1 - K / 256) are at or above it.
    uint32_t lo = 1;
    if (min(nblk, kStreamThreads) >= K) {
        uint32_t v[PER], least = 0xffffffffu, hi = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            v[j] = t.thread_max[lane + 32 * j];
            if (v[j]) least = min(least, v[j]);
            hi = max(hi, v[j]);
        }
        lo = __reduce_min_sync(0xffffffffu, least);
        hi = __reduce_max_sync(0xffffffffu, hi) + 1;
        const int most = K + K / 8 + 4;
        while (hi - lo > 1) {
            const uint32_t mid = lo + (hi - lo) / 2;
            int n = 0;
#pragma unroll
            for (int j = 0; j < PER; ++j) n += v[j] >= mid;
            n = __reduce_add_sync(0xffffffffu, n);
            if (n >= K) {
                lo = mid;
                if (n <= most) break;
            } else {
                hi = mid;
            }
        }
    }
    for (int b0 = 1; b0 <= nblk; b0 += 32 * kStreamThreads) {
        uint32_t hit = 0;
        for (int j = 0, b = b0 + tid; j < 32 && b <= nblk; ++j, b += kStreamThreads)
            hit |= static_cast<uint32_t>(keys[b] >= lo) << j;
        if (__any_sync(0xffffffffu, hit != 0)) {
            int at = warp_places(__popc(hit), &t.n_sel);
            for (; hit; hit &= hit - 1, ++at)
                if (at < kSelCap) t.sel[at] = b0 + tid + (__ffs(hit) - 1) * kStreamThreads;
        }
    }
    consumers_sync();
    int n_sel = t.n_sel, need = 0x7fffffff, strict = 0x7fffffff;  // sel[strict ..]: blocks whose maximum is lo, in order
    if (n_sel > kSelCap) {
        // Ties at the threshold (a mask that leaves fewer than K tokens): the blocks above
        // it, and the first blocks that reach it, as many as can matter.
        consumers_sync();
        if (tid == 0) t.n_sel = 0;
        consumers_sync();
        for (int b = 1 + tid; b <= nblk; b += kStreamThreads) {
            if (keys[b] > lo) {
                const int i = atomicAdd(&t.n_sel, 1);
                if (i < kSelCap) t.sel[i] = b;
            }
        }
        consumers_sync();
        strict = t.n_sel;
        need = K - strict;
        if (strict < K) {
            if (tid < 32) {
                int have = 0;
                for (int b0 = 1; b0 <= nblk && have < need; b0 += 32) {
                    const bool tie = b0 + lane <= nblk && keys[b0 + lane] == lo;
                    const unsigned m = __ballot_sync(0xffffffffu, tie);
                    const int at = have + __popc(m & ((1u << lane) - 1u));
                    if (tie && at < need) t.sel[strict + at] = b0 + lane;
                    have += __popc(m);
                }
                if (lane == 0) t.n_tied = min(have, need);
            }
            consumers_sync();
            n_sel = strict + t.n_tied;
        } else {
            n_sel = kSelCap + 1;  // more than K blocks above the K-th thread maximum: the slow way
        }
    }
    if (n_sel <= kSelCap) {
        // Four threads a block, one vector each (re-read from L2); the elements at or above the threshold.
        const float floor = lo == 1 ? kNegInf : BK::value(lo);
        const uint4* body = reinterpret_cast<const uint4*>(s.body);
        constexpr int TURNS = kSelCap * kBlockVec / kStreamThreads;
        uint4 w[TURNS];
        int vec[TURNS];
#pragma unroll
        for (int q = 0; q < TURNS; ++q) {  // every turn's load goes out before the first is looked at
            const int j = (q * kStreamThreads + tid) / kBlockVec;
            vec[q] = j < n_sel ? (t.sel[j] - 1) * kBlockVec + (tid & (kBlockVec - 1)) : s.nv;
            w[q] = RowMath<ES>::pad();
            if (vec[q] < s.nv) w[q] = ld_global_v4(body + vec[q]);
        }
#pragma unroll
        for (int q = 0; q < TURNS; ++q) {
            if (q * kStreamThreads >= n_sel * kBlockVec) break;
            uint32_t hit = 0, tie = 0;
#pragma unroll
            for (int e = 0; e < EPV / 2; ++e) {
                float lo2, hi2;
                f2_unpack(vec_pair<ES>(w[q], e), lo2, hi2);
                hit |= static_cast<uint32_t>(lo2 >= floor) << 2 * e | static_cast<uint32_t>(hi2 >= floor) << (2 * e + 1);
                tie |= static_cast<uint32_t>(lo2 == floor) << 2 * e | static_cast<uint32_t>(hi2 == floor) << (2 * e + 1);
            }
            if (vec[q] >= s.nv) hit = tie = 0;
            if (strict != 0x7fffffff) {
                // an equal one counts only if fewer than `need` come before it: those of its block's
                // earlier vectors, and one at least in each tied block before
                int sum = __popc(tie);
#pragma unroll
                for (int off = 1; off < kBlockVec; off <<= 1) {
                    const int o = __shfl_up_sync(0xffffffffu, sum, off, kBlockVec);
                    if ((tid & (kBlockVec - 1)) >= off) sum += o;
                }
                int room = need - (sum - __popc(tie)) - max(0, (q * kStreamThreads + tid) / kBlockVec - strict);
                for (uint32_t m = tie; m; m &= m - 1)
                    if (--room < 0) hit &= ~(m & -m);
            }
            if (__any_sync(0xffffffffu, hit != 0)) {
                int at = warp_places(__popc(hit), &t.n_list);
                const uint32_t col = static_cast<uint32_t>(s.col0) + static_cast<uint32_t>(vec[q]) * EPV;
#pragma unroll
                for (int e = 0; e < EPV; ++e) {
                    if (!(hit >> e & 1u)) continue;
                    float lo2, hi2;
                    f2_unpack(vec_pair<ES>(w[q], e / 2), lo2, hi2);
                    const uint32_t key = key_of(e & 1 ? hi2 : lo2);
                    if (at < kListCap) t.list[at] = (static_cast<unsigned long long>(key) << 32) | ~(col + e);
                    ++at;
                }
            }
        }
        if (tid < s.h + s.t) {
            const int64_t col = tid < s.h ? tid : s.tail_col + (tid - s.h);
            const float f = load_scalar<ES>(s.rowp + col * ES);
            if (f >= floor) {
                const int at = atomicAdd(&t.n_list, 1);
                if (at < kListCap)
                    t.list[at] = (static_cast<unsigned long long>(key_of(f)) << 32) | ~static_cast<uint32_t>(col);
            }
        }
        consumers_sync();
        if (t.n_list <= kListCap) return t.n_list;
    }
    top_list_exact<ES>(s, keys, K, t);
    return min(t.n_list, kListCap);
}

template <int ES, bool ENT, bool TOPK>
__global__ void __launch_bounds__(kStreamBlock, 3) logprobs_kernel(const LogprobParams p) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ StreamBars bars;
    __shared__ StatExchange ex;
    __shared__ TopScratch top;
    __shared__ float4 fin;
    using KeyT = typename BlockKey<ES>::type;
    unsigned char* ring = smem;
    KeyT* keys = reinterpret_cast<KeyT*>(smem + p.src.stages * kStreamStageBytes);

    const int tid = threadIdx.x, k = p.src.k;
    const int rank = k > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int64_t cid = blockIdx.x / k, ncl = gridDim.x / k;
    const int64_t n_it = p.src.N > cid ? (p.src.N - 1 - cid) / ncl + 1 : 0;
    stream_init(bars, p.src.stages);
    griddep_launch_dependents();  // programmatic dependent launch: no global access before the wait
    griddep_wait();
    __syncthreads();
    if (k > 1) cluster_sync();  // every CTA's shared memory is there to be written to

    bool bad = false, aborted = false;
    if (tid >= kStreamThreads) {
        stream_produce<ES>(p.src, bars, ring, 1, cid, ncl, rank, k > 1 ? (TOPK ? 3 : 1) : 0);
    } else {
        StreamPos pos{0, 0, false};
        Slice s = slice_of<ES>(p.src, cid, rank);
        uint32_t parity = 0;
        int64_t y_next = p.src.labels && n_it > 0 ? __ldg(p.src.labels + cid) : 0;
        for (int64_t it = 0; it < n_it; ++it) {
            const int64_t row = cid + it * ncl;
            const int64_t y = y_next;
            if (p.src.labels && it + 1 < n_it) y_next = __ldg(p.src.labels + row + ncl);
            if (!stream_row_valid(y, p.src)) {
                bad |= y != p.src.ignore_index;
                if (rank == 0) {
                    if (tid == 0) {
                        if (p.logp) p.logp[row] = 0.f;
                        if (p.entropy) p.entropy[row] = 0.f;
                        if (p.lse) p.lse[row] = 0.f;
                        if (p.stats) p.stats[row] = make_float2(0.f, 0.f);
                    }
                    if (TOPK) {
                        for (int i = tid; i < p.top_k; i += kStreamThreads) {
                            p.top_lp[row * p.top_k + i] = 0.f;
                            p.top_ids[row * p.top_k + i] = -1;
                        }
                    }
                }
                continue;
            }
            move_slice<ES>(p.src, row, rank, s);
            float x_y = 0.f;
            if (tid == 0 && rank == 0 && p.logp) x_y = load_scalar<ES>(s.rowp + y * ES);
            RunStat<ENT, false> st(p.scale);
            float most = kNegInf;  // of the thread's blocks
            for (int c0 = 0; c0 < s.nv; c0 += kStreamChunk) {
                const int nl = min(kStreamChunk, s.nv - c0);
                uint4 v[kBlockVec];
                stream_chunk(p.src, bars, ring, pos, [&](const unsigned char* stage) {
                    if constexpr (TOPK) load_block<ES>(stage, nl, v);
                    else load_strided<ES>(stage, nl, v);
                });
                const float bmax = st.template add_vecs<ES>(v, p.scale);
                if (TOPK) {
                    if (tid * kBlockVec < nl) keys[1 + c0 / kBlockVec + tid] = static_cast<KeyT>(BlockKey<ES>::of(bmax));
                    most = fmaxf(most, bmax);
                }
            }
            if (s.h + s.t > 0 && tid < 32) {  // the head's and the tail's scalars, one a lane
                float e = kNegInf;
                if (tid < s.h + s.t) e = load_scalar<ES>(s.rowp + (tid < s.h ? tid : s.tail_col + (tid - s.h)) * ES);
                st.add(e, p.scale);
                if (TOPK) {
                    const float hm = warp_max_redux(tid < s.h ? e : kNegInf), tm = warp_max_redux(tid < s.h ? kNegInf : e);
                    if (tid == 0) {
                        keys[0] = s.h > 0 ? BlockKey<ES>::of(hm) : 0;
                        keys[1 + (s.nv + kBlockVec - 1) / kBlockVec] = s.t > 0 ? BlockKey<ES>::of(tm) : 0;
                    }
                }
            } else if (TOPK && tid == 0) {
                keys[0] = keys[1 + (s.nv + kBlockVec - 1) / kBlockVec] = 0;
            }
            if (TOPK) {
                top.thread_max[tid] = tid * kBlockVec < s.nv ? BlockKey<ES>::of(most) : 0u;
                if (tid == 0) top.n_sel = top.n_list = 0;
            }
            stat_publish(st, ex, parity);
            consumers_sync();
            if (tid < 32) stat_collect(st, ex, parity, p.scale);
            if (k > 1) {
                if (tid < 32) stat_send(st, ex, parity, k, rank);
                cluster_sync_converged();
                if (tid < 32) stat_merge(st, ex, parity, k, p.scale);
            }
            parity ^= 1u;
            if (tid < 32) {  // the row's results; the rest of the CTA goes on to the top tokens
                st.correct(p.scale);
                const float ln_s = logf(st.s);
                const bool empty = st.s == 0.f;
                if (tid == 0) {
                    if (TOPK) fin = make_float4(st.m, ln_s, st.s, 0.f);
                    if (rank == 0 && !pos.aborted) {
                        if (p.logp) p.logp[row] = empty ? kNegInf : (x_y - st.m) * p.inv_t - ln_s;
                        if (ENT) {
                            const float h = ln_s - st.a * kLn2 / st.s;
                            p.entropy[row] = empty || h < 0.f ? 0.f : h;
                        }
                        if (p.lse) p.lse[row] = empty ? kNegInf : fmaf(st.m, p.inv_t, ln_s);
                        if (p.stats) p.stats[row] = make_float2(empty ? kNegInf : st.m, ln_s);
                    }
                }
            }
            if constexpr (TOPK) {
                const int K = p.top_k;
                const int n = top_list<ES>(s, keys, K, top);
                const float4 f = fin;  // (m, ln S, S): written before the barriers of top_list
                const bool none = !(f.z == f.z);  // a NaN or +inf in the row: no order to speak of
                const bool empty = f.z == 0.f;
                float* olp = p.top_lp + row * K;
                int32_t* oid = p.top_ids + row * K;
                auto write = [&](int r, unsigned long long item) {
                    if (pos.aborted || none) return;
                    olp[r] = empty ? kNegInf : (float_of_key(static_cast<uint32_t>(item >> 32)) - f.x) * p.inv_t - f.y;
                    oid[r] = static_cast<int32_t>(~static_cast<uint32_t>(item));
                };
                // Ranks within this CTA's list: `ways` neighbouring threads an item, each comparing it with
                // its share of the list, two items a 16-byte read.
                if (k > 1) {
                    if (tid < K) top.best[tid] = 0ull;
                    consumers_sync();
                }
                const int ways = n <= kStreamThreads / 8 ? 8 : n <= kStreamThreads / 4 ? 4 : n <= kStreamThreads / 2 ? 2 : 1;
                const int part = tid & (ways - 1);
                for (int i0 = 0; i0 < n; i0 += kStreamThreads / ways) {
                    const int i = i0 + tid / ways;
                    const unsigned long long item = i < n ? top.list[i] : ~0ull;
                    int r = 0;
                    for (int j = 2 * part; j < n; j += 2 * ways) {
                        const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(top.list + j);
                        r += o.x > item;
                        if (j + 1 < n) r += o.y > item;
                    }
                    for (int off = 1; off < ways; off <<= 1) r += __shfl_xor_sync(0xffffffffu, r, off);
                    if (i < n && part == 0 && r < K) {
                        if (k > 1) top.best[r] = item;
                        else write(r, item);
                    }
                }
                if (k > 1) {
                    // The cluster's lists, each in order: an item's rank is the sum of its places in them,
                    // one thread an item and list.  They are copied here first when there is room.
                    cluster_sync_converged();  // every CTA's best are in place
                    const bool copy = K * k <= kListCap;
                    if (copy) {
                        for (int i = tid; i < K * k; i += kStreamThreads) {
                            const uint32_t from = mapa_u32(top.best, static_cast<uint32_t>(i / K)) + (i % K) * 8;
                            asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(top.list[i]) : "r"(from) : "memory");
                        }
                    }
                    consumers_sync();
                    for (int i0 = 0; i0 < K * k; i0 += kStreamThreads) {
                        const int i = i0 + tid;
                        const int o = i & (k - 1);
                        const unsigned long long item = i < K * k ? top.best[i / k] : 0ull;
                        int a = 0, b = item ? K : 0;  // of list o: before a larger, from b on not
                        const uint32_t remote = mapa_u32(top.best, static_cast<uint32_t>(o));
                        while (a < b) {
                            const int mid = (a + b) / 2;
                            unsigned long long v;
                            if (copy) v = top.list[o * K + mid];
                            else asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote + mid * 8) : "memory");
                            if (v > item) a = mid + 1;
                            else b = mid;
                        }
                        __syncwarp();
                        for (int off = 1; off < k; off <<= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
                        if (o == 0 && item && a < K) write(a, item);
                    }
                    cluster_sync_converged();  // every CTA has read them
                }
                if (none && rank == 0) {
                    for (int i = tid; i < K; i += kStreamThreads) {
                        olp[i] = f.z;
                        oid[i] = -1;
                    }
                }
                consumers_sync();  // the keys and lists may be overwritten
            }
        }
        aborted = pos.aborted;
    }
    // The error word: every CTA adds its bits; the last one publishes and resets them.
    __syncthreads();
    if (tid == 0) {
        unsigned e = 0;
        if (aborted || stream_aborted(bars)) e |= FOAK_ERRBIT_TIMEOUT;
        if (bad) e |= FOAK_ERRBIT_LABEL_RANGE;
        if (e) atomicOr(&p.ws->err, e);
        if (atom_add_acq_rel_gpu(&p.ws->done, 1u) == gridDim.x - 1) {
            e = atomicExch(&p.ws->err, 0u);
            atomicExch(&p.ws->done, 0u);
            if (p.err) *p.err = static_cast<int32_t>(e);
        }
    }
    if (k > 1) cluster_sync_converged();  // no CTA leaves while its shared memory may be read
}

std::mutex g_lp_mu;
std::map<std::pair<int, const void*>, size_t> g_lp_attr;  // (device, kernel): dynamic shared memory allowed

template <int ES, bool ENT, bool TOPK>
cudaError_t launch_typed(LogprobParams prm, cudaStream_t stream) {
    auto* kern = &logprobs_kernel<ES, ENT, TOPK>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    StreamSrc& s = prm.src;
    const int sms = device_sm_count();
    const int64_t nb = s.V * ES / 16 + 1;
    // Few rows: a cluster per row, as long as its CTAs are all on SMs of their own and
    // have at least half a chunk each.
    int k = kStreamMaxCluster;
    while (k > 1 && (s.N * k > sms || 2 * nb < static_cast<int64_t>(k) * kStreamChunk)) k /= 2;
    set_cluster(s, k);
    const int64_t nblk = ((nb + kBlockVec - 1) / kBlockVec + s.k - 1) / s.k + 3;
    const size_t key_bytes = TOPK ? (static_cast<size_t>(nblk) * sizeof(typename BlockKey<ES>::type) + 127) / 128 * 128 : 0;
    // Three CTAs an SM when each gets a ring of three stages, else two.
    const size_t fixed = 1024 + sizeof(StreamBars) + sizeof(StatExchange) + sizeof(TopScratch) + 256 + key_bytes;
    int per_sm = 3;
    while (per_sm > 1 && (228 * 1024) / per_sm < fixed + 3 * kStreamStageBytes) --per_sm;
    const size_t room = std::min<size_t>((228 * 1024) / per_sm, 227 * 1024) - fixed;
    s.stages = static_cast<int>(std::min<size_t>(kStreamMaxStages, room / kStreamStageBytes));
    if (s.stages < 1) return cudaErrorInvalidValue;
    const size_t smem = static_cast<size_t>(s.stages) * kStreamStageBytes + key_bytes;
    {
        std::lock_guard<std::mutex> lock(g_lp_mu);
        size_t& set = g_lp_attr[std::make_pair(dev, reinterpret_cast<const void*>(kern))];
        if (set < smem) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
            if (e != cudaSuccess) return e;
            set = smem;
        }
    }
    const int64_t clusters = std::max<int64_t>(1, std::min<int64_t>(s.N, static_cast<int64_t>(sms) * per_sm / s.k));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * s.k), 1, 1);
    cfg.blockDim = dim3(kStreamBlock, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0] = pdl_attribute();
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(s.k);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = s.k > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, prm);
}

}  // namespace

cudaError_t launch_logprobs(int es, const void* x, int64_t ld, const int64_t* labels, int64_t N, int64_t V,
                            int64_t ignore_index, float temperature, int top_k, float* logp, float* entropy, float* lse,
                            float* stats, float* top_lp, int32_t* top_ids, int32_t* err, CeWsHeader* ws,
                            cudaStream_t stream) {
    LogprobParams p = {};
    p.src.x = static_cast<const char*>(x);
    p.src.ld = ld;
    p.src.labels = labels;
    p.src.N = N;
    p.src.V = V;
    p.src.ignore_index = ignore_index;
    p.src.wait_ns = test_wait_limit_ns();
    p.src.skip_load_row = test_skip_load_row();
    p.inv_t = 1.f / temperature;
    p.scale = exp_scale(temperature);
    p.top_k = top_k;
    p.logp = logp;
    p.entropy = entropy;
    p.lse = lse;
    p.stats = reinterpret_cast<float2*>(stats);
    p.top_lp = top_lp;
    p.top_ids = top_ids;
    p.err = err;
    p.ws = ws;
    if (es == 2) {
        if (top_k > 0) return entropy ? launch_typed<2, true, true>(p, stream) : launch_typed<2, false, true>(p, stream);
        return entropy ? launch_typed<2, true, false>(p, stream) : launch_typed<2, false, false>(p, stream);
    }
    if (top_k > 0) return entropy ? launch_typed<4, true, true>(p, stream) : launch_typed<4, false, true>(p, stream);
    return entropy ? launch_typed<4, true, false>(p, stream) : launch_typed<4, false, false>(p, stream);
}

}  // namespace foak
