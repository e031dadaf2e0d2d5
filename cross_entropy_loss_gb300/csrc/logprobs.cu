// Log probability of a given token, entropy and the K most likely tokens of every row
// of logits -- what a server answering with log probabilities, a policy-gradient step
// or a teacher writing down its distribution takes from the LM head.  With z = x / T:
//
//   m = max_j x_j     S = sum_j e^{(x_j - m) / T}     A = sum_j e^{(x_j - m) / T} (x_j - m) / T
//   lse = m / T + ln S     logp_j = (x_j - m) / T - ln S     H = ln S - A / S
//
// One read of the row gives m, S and A (running sums per thread, rescaled at a new
// maximum).  The top K come out of the same read: a thread's 64-byte block of a chunk
// has one maximum, which the sums need anyway and which is kept.  Blocks (32 elements) are
// contiguous, so the K largest blocks by (maximum, lower index first) hold the K largest
// elements by (value, lower index first): with a total order an element outside those
// blocks has K larger ones before it.  A row's end, by one of the
// CTA's three closing warps while the others are on the next rows, is
//
//   1. a threshold that at least K blocks reach, from the 256 consumer threads' maxima;
//   2. the blocks at or above it, re-read (from L2: the row just went through), and their
//      elements at or above the threshold put on a list;
//   3. the list put in order, in registers.
//
// Rows go to CTAs round-robin; when there are few a cluster shares each row, joins its
// sums and lists through distributed shared memory, and ranks every CTA's K candidates
// against the others'.
//
// Measured, with entropy, bf16 unless said: 8192 x 128256, K = 0, 20, 128: 307, 357, 404 us
// (6.85, 5.9, 5.2 TB/s); 4096 x 32000, K = 0, 5: 48.5 and 66; 2048 x 128256 fp32, K = 64: 188 (5.6
// TB/s); 1 x 128256, K = 0, 20: 6.6 and 14; 64 x 128256 under a mask, K = 20: 22.  HBM bounds the
// long rows.  With top tokens a row's end is some 10000 cycles alone, three times that
// beside warps that sum: short rows and few rows pay for it.
#include <algorithm>

#include "row_stream.cuh"

namespace foak {

namespace {

constexpr int kListCap = 384;   // listed elements of a row (or of a CTA's share of it): at least kTopKMax
constexpr int kSelCap = 320;    // blocks they are taken from
constexpr int kAll = 0x7fffffff;
constexpr int kThreads = 256;   // consumers
using Sh = Shape<kThreads>;
static_assert(kTopKMaxVocab <= static_cast<int64_t>(kRunVec<kThreads>) * 4, "rows with top tokens are one run of chunks");
constexpr int kBodyAt = 8;      // place of the first body block's maximum; before it the head's and the tail's
// Closing warps of a CTA.  The work on a row's top tokens is a chain of 10000 cycles or more,
// so three take rows in turn (8192 x 128256, K = 128: two with two CTAs an SM 464 us, three
// with three 454, four 487); without top tokens one keeps up.  At three CTAs an SM a thread
// has 56 registers, and their code spills (about 320 bytes of stores in close_rows).
template <bool TOPK>
constexpr int kClosers = TOPK ? 3 : 1;

struct LogprobParams {
    StreamSrc src;
    float inv_t;       // 1 / T
    ExpScale scale;
    int top_k;
    int max_stride;    // places of a row's block maxima in shared memory
    int max_bytes;     // of all buffers'; a shared row's lists follow
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
// A block: 32 elements.  Its maximum is kept as the float it is (bf16: its upper half), NaN
// for a block that is not there.
template <int ES>
struct Block {
    using type = uint32_t;
    static constexpr int kVec = 8;         // its 16-byte vectors
    static constexpr int kPieces = 2;      // its 64-byte pieces, a thread's share of a chunk
    static constexpr uint32_t kNone = 0x7fffffffu;
    static __device__ __forceinline__ uint32_t pack(float f) { return __float_as_uint(f); }
    static __device__ __forceinline__ float value(uint32_t v) { return __uint_as_float(v); }
};
template <>
struct Block<2> {
    using type = uint16_t;
    static constexpr int kVec = 4;
    static constexpr int kPieces = 1;
    static constexpr uint32_t kNone = 0x7fffu;
    static __device__ __forceinline__ uint16_t pack(float f) { return static_cast<uint16_t>(__float_as_uint(f) >> 16); }
    static __device__ __forceinline__ float value(uint32_t v) { return __uint_as_float(v << 16); }
};
// Keys of the thread maxima: of bf16 the upper half alone, whose lower half is constant.
template <int ES>
__device__ __forceinline__ uint32_t short_key(float f) {
    return ES == 2 ? key_of(f) >> 16 : key_of(f);
}
template <int ES>
__device__ __forceinline__ float float_of_short_key(uint32_t k) {
    if constexpr (ES == 4) return float_of_key(k);
    else return float_of_key(k >> 15 ? k << 16 : k << 16 | 0xffffu);  // a negative number's lower half is ones
}

// A closing warp's scratch.
struct TopScratch {
    alignas(16) unsigned long long list[kListCap];  // (key << 32) | ~column
    uint16_t sel[kSelCap];                          // the chosen blocks
    float floor;                                    // a threshold on its way to top_list_again
};

__device__ __forceinline__ unsigned lanes_below() { return (1u << (threadIdx.x & 31)) - 1u; }

// Block `id` of the slice: 0 the head scalars, 1 .. nblk the body's blocks, nblk + 1 the tail scalars.
template <int ES>
struct BlockElements {
    static constexpr int EPV = 16 / ES;
    static constexpr int VEC = Block<ES>::kVec;
    static constexpr int N = VEC * EPV;
    uint32_t w[VEC * 4];  // the elements as they lie in memory
    int n;
    int64_t col;

    __device__ __forceinline__ void load(const Slice& s, int id, int nblk) {
#pragma unroll
        for (int i = 0; i < VEC * 4; ++i) w[i] = 0;
        if (id > 0 && id <= nblk) {
            const int v0 = (id - 1) * VEC;
            const int nv = min(VEC, s.nv - v0);
            col = s.col0 + static_cast<int64_t>(v0) * EPV;
            n = nv * EPV;
            const uint4* v = reinterpret_cast<const uint4*>(s.body) + v0;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
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

// Everything from here to the kernel is one warp's work.

// The slow way to the list, for rows in which the fast one meets more blocks or elements
// than it has room for (many equal values, or a share of few blocks): exact bisections,
// first for the K-th largest block by (maximum, lower index first), then, if need be, for
// the K-th largest element.  Up to K blocks, all of them are taken.
template <int ES>
__device__ __noinline__ int top_list_exact(const Slice s, const typename Block<ES>::type* maxima, int K, TopScratch& t) {
    const int lane = threadIdx.x & 31;
    const int nblk = (s.nv + Block<ES>::kVec - 1) / Block<ES>::kVec;
    const int nreal = nblk + (s.h > 0) + (s.t > 0);
    auto key = [&](int b) -> uint32_t {
        const float f = Block<ES>::value(maxima[b == 0 ? 0 : b > nblk ? 1 : kBodyAt - 1 + b]);
        return f == f ? key_of(f) : 0u;
    };
    // ---- the blocks: keys above lo, and of those equal to lo the ids up to last
    uint32_t lo = 1;
    int last = kAll;
    if (nreal > K) {
        uint32_t hi = 0xffffffffu;   // above every key
        int c_lo = nreal, c_hi = 0;  // blocks at or above lo and hi
#pragma unroll 1
        while (hi - lo > 1 && c_lo > kSelCap) {
            const uint32_t mid = lo + (hi - lo) / 2;
            int n = 0;
#pragma unroll 1
            for (int b = lane; b < nblk + 2; b += 32) n += key(b) >= mid;
            n = __reduce_add_sync(0xffffffffu, n);
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
#pragma unroll 1
            while (j1 - j0 > 1) {
                const int mid = j0 + (j1 - j0) / 2;
                int n = 0;
#pragma unroll 1
                for (int b = lane; b <= mid; b += 32) n += key(b) == lo;
                if (__reduce_add_sync(0xffffffffu, n) >= need) j1 = mid;
                else j0 = mid;
            }
            last = j1;
        }
    }
    int n_sel = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < nblk + 2; b0 += 32) {
        const int b = b0 + lane;
        const uint32_t k = b < nblk + 2 ? key(b) : 0;
        const bool hit = k > lo || (k == lo && b <= last);
        const unsigned m = __ballot_sync(0xffffffffu, hit);
        const int at = n_sel + __popc(m & lanes_below());
        if (hit && at < kSelCap) t.sel[at] = static_cast<uint16_t>(b);
        n_sel += __popc(m);
    }
    n_sel = min(n_sel, kSelCap);
    __syncwarp();
    // ---- their elements: a block a lane and turn, read again for every count
    auto for_each = [&](auto&& f) {
#pragma unroll 1
        for (int i0 = 0; i0 < n_sel; i0 += 32) {
            BlockElements<ES> el;
            el.n = 0;
            el.col = 0;
            if (i0 + lane < n_sel) el.load(s, t.sel[i0 + lane], nblk);
#pragma unroll
            for (int e = 0; e < BlockElements<ES>::N; ++e) f(el.item(e));
        }
    };
    auto at_least = [&](unsigned long long f) {
        int n = 0;
        for_each([&](unsigned long long it) { n += it >= f; });
        return __reduce_add_sync(0xffffffffu, n);
    };
    // every count is at least K at b0 (or takes every element) and less than K at b1
    unsigned long long b0 = static_cast<unsigned long long>(lo) << 32, b1 = ~0ull;
    if (at_least(b0) > kListCap) {
#pragma unroll 1
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
    int n = 0;
    for_each([&](unsigned long long it) {
        const bool hit = it >= b0;
        const unsigned m = __ballot_sync(0xffffffffu, hit);
        const int at = n + __popc(m & lanes_below());
        if (hit && at < kListCap) t.list[at] = it;
        n += __popc(m);
    });
    __syncwarp();
    return min(n, kListCap);
}

// Of the elements of a 16-byte word group: a bit for each that is >= floor (or == floor).
// bf16: bit k the lower and bit 16 + k the upper element of word k; fp32: bit k element k.
template <int ES, bool EQUAL, int WORDS>
__device__ __forceinline__ uint32_t hit_bits(const uint32_t (&w)[WORDS], float floor) {
    uint32_t bits = 0;
    if constexpr (ES == 2) {
        const __nv_bfloat162 f = __float2bfloat162_rn(floor);
#pragma unroll
        for (int k = 0; k < WORDS; ++k) {
            const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w[k]);
            bits |= (EQUAL ? __heq2_mask(x, f) : __hge2_mask(x, f)) & (0x10001u << k);
        }
    } else {
#pragma unroll
        for (int k = 0; k < WORDS; ++k) {
            const float x = __uint_as_float(w[k]);
            bits |= (EQUAL ? x == floor : x >= floor) ? 1u << k : 0u;
        }
    }
    return bits;
}
template <int ES>
__device__ __forceinline__ int element_of_bit(int b) {
    return ES == 2 ? (b & 15) << 1 | b >> 4 : b;
}
// the bits of the first n elements
template <int ES>
__device__ __forceinline__ uint32_t first_bits(int n) {
    if constexpr (ES == 2) return ((1u << (n + 1) / 2) - 1u) | ((1u << n / 2) - 1u) << 16;
    else return (1u << n) - 1u;
}

// The blocks of the body whose maximum reaches the floor (above: is above it) onto sel, 16
// bytes of maxima a lane and turn.  Returns how many, or some number above kSelCap.
template <int ES>
__device__ __forceinline__ int blocks_from(const typename Block<ES>::type* maxima, int nblk, float floor, bool above,
                                           uint16_t* sel) {
    constexpr int PACK = 16 / sizeof(typename Block<ES>::type);
    const int lane = threadIdx.x & 31;
    const uint4* mv = reinterpret_cast<const uint4*>(maxima + kBodyAt);
    int n = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < nblk && n <= kSelCap; b0 += 32 * PACK) {
        const int b = b0 + lane * PACK;
        uint32_t hit = 0;
        if (b < nblk) {
            const uint4 q = mv[b / PACK];
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
            hit = hit_bits<ES, false>(w, floor);
            if (above) hit &= ~hit_bits<ES, true>(w, floor);
            if (nblk - b < PACK) hit &= first_bits<ES>(nblk - b);
        }
#pragma unroll 1
        for (unsigned m = __ballot_sync(0xffffffffu, hit != 0); m; m = __ballot_sync(0xffffffffu, hit != 0)) {
            const int at = n + __popc(m & lanes_below());
            if (hit && at < kSelCap) sel[at] = static_cast<uint16_t>(1 + b + element_of_bit<ES>(__ffs(hit) - 1));
            hit &= hit - 1;
            n += __popc(m);
        }
    }
    __syncwarp();
    return n;
}
// The same out of line, for the ways that few rows take.
template <int ES>
__device__ __noinline__ int blocks_again(const typename Block<ES>::type* maxima, int nblk, float floor, bool above,
                                         uint16_t* sel) {
    return blocks_from<ES>(maxima, nblk, floor, above, sel);
}
// A higher threshold for a row in which more blocks than sel has room for are above `floor`:
// K blocks reach it, and no more than `most` unless they are equal there.
template <int ES>
__device__ __noinline__ float blocks_floor(const typename Block<ES>::type* maxima, int nblk, float floor, int K,
                                           int most) {
    constexpr int PACK = 16 / sizeof(typename Block<ES>::type);
    const int lane = threadIdx.x & 31;
    const uint4* mv = reinterpret_cast<const uint4*>(maxima + kBodyAt);
    uint32_t lo = short_key<ES>(floor), hi = short_key<ES>(__uint_as_float(0x7f800000u)) + 1u;
#pragma unroll 1
    while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        const float f = float_of_short_key<ES>(mid);
        int n = 0;
#pragma unroll 1
        for (int b = lane * PACK; b < nblk; b += 32 * PACK) {
            const uint4 q = mv[b / PACK];
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
            uint32_t hit = hit_bits<ES, false>(w, f);
            if (nblk - b < PACK) hit &= first_bits<ES>(nblk - b);
            n += __popc(hit);
        }
        n = __reduce_add_sync(0xffffffffu, n);
        if (n >= K) {
            lo = mid;
            if (n <= most) break;
        } else {
            hi = mid;
        }
    }
    return float_of_short_key<ES>(lo);
}

// The first elements equal to the floor onto the list, which has n, until it has K: the
// blocks whose maximum reaches the floor one by one, an element a lane.  (A block whose
// maximum is the floor has one at least, and there are fewer than K others.)
template <int ES>
__device__ __noinline__ int list_equal(const Slice s, const typename Block<ES>::type* maxima, int nblk, float floor, int K,
                                       int n, TopScratch& t) {
    constexpr int EPV = 16 / ES;
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int b0 = 0; b0 < nblk + 2 && n < K; b0 += 32) {
        const int b = b0 + lane;
        const bool may = b < nblk + 2 && Block<ES>::value(maxima[b == 0 ? 0 : b > nblk ? 1 : kBodyAt - 1 + b]) >= floor;
#pragma unroll 1
        for (unsigned m = __ballot_sync(0xffffffffu, may); m && n < K; m &= m - 1) {
            const int id = b0 + __ffs(m) - 1, v0 = (id - 1) * Block<ES>::kVec;
            const int64_t col = lane + (id == 0 ? 0 : id > nblk ? s.tail_col : s.col0 + static_cast<int64_t>(v0) * EPV);
            const bool there = lane < (id == 0 ? s.h : id > nblk ? s.t : min(Block<ES>::kVec, s.nv - v0) * EPV);
            float f = 0.f;
            if (there) f = load_scalar<ES>(s.rowp + col * ES);
            const bool hit = there && f == floor;
            const unsigned hits = __ballot_sync(0xffffffffu, hit);
            const int at = n + __popc(hits & lanes_below());
            if (hit && at < K) t.list[at] = (static_cast<unsigned long long>(key_of(f)) << 32) | ~static_cast<uint32_t>(col);
            n += __popc(hits);
        }
    }
    __syncwarp();
    return min(n, K);
}

// The elements at or above the floor (above: above it) of the chosen blocks and of the head
// and tail onto the list.  Returns how many there are, which may be more than it takes.
template <int ES>
__device__ __forceinline__ int list_from(const Slice& s, float floor, bool above, int n_sel, TopScratch& t) {
    using B = Block<ES>;
    constexpr int EPV = 16 / ES;
    const int lane = threadIdx.x & 31;
    const uint4* body = reinterpret_cast<const uint4*>(s.body);
    int n = 0;
    // a 64-byte piece a lane and turn (re-read from L2)
#pragma unroll 1
    for (int i0 = 0; i0 < n_sel * B::kPieces; i0 += 32) {
        const int i = i0 + lane, j = i / B::kPieces;
        const bool there = j < n_sel;
        const int vec = there ? (t.sel[j] - 1) * B::kVec + i % B::kPieces * kBlockVec : 0;
        const int nv = there ? min(kBlockVec, s.nv - vec) : 0;
        uint32_t w[4 * kBlockVec];
#pragma unroll
        for (int q = 0; q < kBlockVec; ++q) {
            uint4 r = RowMath<ES>::pad();
            if (q < nv) r = ld_global_v4(body + vec + q);
            w[4 * q] = r.x, w[4 * q + 1] = r.y, w[4 * q + 2] = r.z, w[4 * q + 3] = r.w;
        }
        uint32_t hit = hit_bits<ES, false>(w, floor);
        if (nv < kBlockVec) hit &= nv > 0 ? first_bits<ES>(nv * EPV) : 0u;
        if (above) hit &= ~hit_bits<ES, true>(w, floor);
        int at = __popc(hit);  // then the places before the lane's
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, at, off);
            if (lane >= off) at += o;
        }
        const int end = n + __shfl_sync(0xffffffffu, at, 31);
        at += n - __popc(hit);
        n = end;
#pragma unroll 1
        for (; hit; hit &= hit - 1, ++at) {
            const int e = element_of_bit<ES>(__ffs(hit) - 1);
            const int64_t col = s.col0 + static_cast<int64_t>(vec) * EPV + e;
            const float f = load_scalar<ES>(s.rowp + col * ES);  // it is in L1
            if (at < kListCap)
                t.list[at] = (static_cast<unsigned long long>(key_of(f)) << 32) | ~static_cast<uint32_t>(col);
        }
    }
    if (s.h + s.t > 0) {
        const int64_t col = lane < s.h ? lane : s.tail_col + (lane - s.h);
        float f = kNegInf;
        if (lane < s.h + s.t) f = load_scalar<ES>(s.rowp + col * ES);
        const bool hit = lane < s.h + s.t && (above ? f > floor : f >= floor);
        const unsigned m = __ballot_sync(0xffffffffu, hit);
        const int at = n + __popc(m & lanes_below());
        if (hit && at < kListCap)
            t.list[at] = (static_cast<unsigned long long>(key_of(f)) << 32) | ~static_cast<uint32_t>(col);
        n += __popc(m);
    }
    __syncwarp();
    return n;
}

// So many blocks or threads at or above a threshold for K tokens will do.
__device__ __forceinline__ int enough(int K) { return K + K / 16 + 4; }

// The list of a row for which a threshold from the threads' maxima is no good.  t.floor is
// that threshold; K elements reach it, if the slice has so many.
template <int ES>
__device__ __noinline__ int top_list_again(const Slice s, const typename Block<ES>::type* maxima, int K, TopScratch& t) {
    const int nblk = (s.nv + Block<ES>::kVec - 1) / Block<ES>::kVec;
    float floor = t.floor;
    // Many blocks reach it because they are equal there (a mask that leaves fewer than K tokens): the
    // elements above it first, then the first ones that are equal.
    bool above = true;
    int n_sel = blocks_again<ES>(maxima, nblk, floor, true, t.sel);
    if (n_sel >= K) {  // not so: K is near the threads' number, or the logits are in no random order
        floor = blocks_floor<ES>(maxima, nblk, floor, K, enough(K));
        n_sel = blocks_again<ES>(maxima, nblk, floor, false, t.sel);
        above = n_sel > kSelCap;
        if (above) n_sel = blocks_again<ES>(maxima, nblk, floor, true, t.sel);
    }
#pragma unroll 1
    while (n_sel <= kSelCap) {
        const int n = list_from<ES>(s, floor, above, n_sel, t);
        if (n <= kListCap) return above && n < K ? list_equal<ES>(s, maxima, nblk, floor, K, n, t) : n;
        if (above) break;
        // Too many elements in a few blocks: perhaps equal ones.
        above = true;
        n_sel = blocks_again<ES>(maxima, nblk, floor, true, t.sel);
        if (n_sel >= K) break;
    }
    return top_list_exact<ES>(s, maxima, K, t);
}

// This CTA's largest elements of its slice onto t.list: at least the min(K, all) largest
// ones, at most kListCap.  Returns how many.  maxima are the blocks' (kBodyAt the first of
// the body; 0 and 1 the head's and tail's), thread_max the keys of the threads'.
template <int ES>
__device__ __noinline__ int top_list(const Slice s, const typename Block<ES>::type* maxima, const uint32_t* thread_max,
                                     int K, TopScratch& t) {
    constexpr int PER = kThreads / 32;
    const int lane = threadIdx.x & 31;
    const int nblk = (s.nv + Block<ES>::kVec - 1) / Block<ES>::kVec;
    // A threshold that K threads' maxima, so K elements, reach: the K-th largest of the 256
    // thread maxima, or a little below it.  Of 64-byte pieces in random order about
    // -256 ln(1 - K / 256) are at or above it.
    float floor = kNegInf;
    if (min((s.nv + kBlockVec - 1) / kBlockVec, kThreads) >= K) {
        uint32_t v[PER], least = 0xffffffffu, hi = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            v[j] = thread_max[lane + 32 * j];
            least = min(least, v[j] - 1u);  // 0, no piece, becomes the largest
            hi = max(hi, v[j]);
        }
        uint32_t lo = __reduce_min_sync(0xffffffffu, least) + 1u;
        hi = __reduce_max_sync(0xffffffffu, hi) + 1u;
#pragma unroll 1
        while (hi - lo > 1) {
            const uint32_t mid = lo + (hi - lo) / 2;
            int n = 0;
#pragma unroll
            for (int j = 0; j < PER; ++j) n += v[j] >= mid;
            n = __reduce_add_sync(0xffffffffu, n);
            if (n >= K) {
                lo = mid;
                if (n <= enough(K)) break;
            } else {
                hi = mid;
            }
        }
        floor = float_of_short_key<ES>(lo);
    }
    if (floor > kNegInf) {
        const int n_sel = blocks_from<ES>(maxima, nblk, floor, false, t.sel);
        if (n_sel <= kSelCap) {
            const int n = list_from<ES>(s, floor, false, n_sel, t);
            if (n <= kListCap) return n;
        }
    }
    if (lane == 0) t.floor = floor;
    __syncwarp();
    return top_list_again<ES>(s, maxima, K, t);
}

// The list in descending order, R items a lane: a bitonic sort in registers, lane l
// holding the places l R .. l R + R - 1; the places from n to 32 R (or the list's end) get 0.
template <int R>
__device__ __noinline__ void sort_list(unsigned long long* list, int n) {
    const int lane = threadIdx.x & 31;
    unsigned long long v[R];
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = r * 32 + lane < n ? list[r * 32 + lane] : 0ull;  // any order will do
#pragma unroll 1
    for (int size = 2; size <= 32 * R; size *= 2) {
#pragma unroll 1
        for (int d = size / (2 * R); d > 0; d /= 2) {  // strides of whole lanes
            const bool larger = ((lane & d) == 0) == ((lane * R & size) == 0 || size == 32 * R);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const unsigned long long o = __shfl_xor_sync(0xffffffffu, v[r], d);
                v[r] = larger == (o > v[r]) ? o : v[r];
            }
        }
#pragma unroll
        for (int stride = R / 2; stride > 0; stride /= 2) {  // and inside a lane
            if (stride >= size) continue;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (r & stride) continue;
                const bool down = ((lane * R + r) & size) == 0 || size == 32 * R;  // this run descends
                const unsigned long long a = v[r], b = v[r + stride];
                const bool swap = down ? a < b : b < a;
                v[r] = swap ? b : a;
                v[r + stride] = swap ? a : b;
            }
        }
    }
    __syncwarp();
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (32 * R <= kListCap || lane * R + r < kListCap) list[lane * R + r] = v[r];
}
// Up to 32 items: each lane counts the larger ones of its own, eight at a time, whose loads
// go out together.
__device__ __forceinline__ void sort_short_list(unsigned long long* list, int n) {
    const int lane = threadIdx.x & 31;
    const unsigned long long mine = lane < n ? list[lane] : 0ull;
    if (lane >= n) list[lane] = 0ull;
    __syncwarp();
    const uint32_t at = smem_u32(list);
    int r = 0;
#pragma unroll 1
    for (int j = 0; j < n; j += 8) {
        unsigned long long v[8];
#pragma unroll
        for (int q = 0; q < 8; q += 2)
            asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(v[q]), "=l"(v[q + 1]) : "r"(at + (j + q) * 8) : "memory");
#pragma unroll
        for (int q = 0; q < 8; ++q) r += v[q] > mine;
    }
    __syncwarp();
    if (lane < n) list[r] = mine;
}
__device__ __forceinline__ void top_ordered(unsigned long long* list, int n) {
    if (n <= 32) sort_short_list(list, n);
    else if (n <= 64) sort_list<2>(list, n);
    else if (n <= 128) sort_list<4>(list, n);
    else if (n <= 256) sort_list<8>(list, n);
    else sort_list<16>(list, n);
    __syncwarp();
}

// A cluster's lists, out of line: rows that have a CTA to themselves do not pay for the code.
//
// This CTA's n largest, in order, into every CTA's `pushed`, which has K places for each.
__device__ __noinline__ void push_list(unsigned long long* best, int n, int K, unsigned long long* pushed, int rank, int k) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int i = n + lane; i < K; i += 32) best[i] = 0ull;
    __syncwarp();
#pragma unroll 1
    for (int i = lane; i < K; i += 32) {
        const unsigned long long v = best[i];
#pragma unroll 1
        for (int o = 0; o < k; ++o) {
            const uint32_t to = mapa_u32(pushed + rank * K + i, static_cast<uint32_t>(o));
            asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(v) : "memory");
        }
    }
}
// An item's rank among the cluster's: the sum of its places in the lists, by a bisection of
// each.  (Looked up in the other CTAs' memory instead of here, 16 rows of 128256 took 27 us at
// K = 65, 23 this way.)
__device__ __noinline__ int pushed_rank(const unsigned long long* pushed, int K, int k, unsigned long long item) {
    int r = 0;
#pragma unroll 1
    for (int o = 0; o < k; ++o, pushed += K) {
        int a = 0, b = K;  // before a larger, from b on not
#pragma unroll 1
        while (a < b) {
            const int mid = (a + b) / 2;
            if (pushed[mid] > item) a = mid + 1;
            else b = mid;
        }
        r += a;
    }
    return r;
}

template <bool TOPK>
constexpr int kLogprobThreads = Sh::kFirstCloser + 32 * kClosers<TOPK>;

// A closing warp's rows.  Not inlined: its registers are not the consumers' concern.
template <int ES, bool ENT, bool TOPK>
__device__ __noinline__ void close_rows(const LogprobParams& p, StreamBars& bars, StatExchange& ex, TopScratch* top,
                                        const uint32_t (*thread_max)[kThreads], const typename Block<ES>::type* maxima,
                                        unsigned char* smem_pushed, int64_t label0) {
    const int lane = threadIdx.x & 31, k = p.src.k;
    const int rank = k > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int64_t cid = blockIdx.x >> p.src.log2_k, ncl = gridDim.x >> p.src.log2_k;
    const int64_t n_it = stream_rows(p.src, cid);
    const int me = (threadIdx.x >> 5) - (Sh::kWarps + 1);  // with several closing warps, buffer `me` is this one's
    RowPos rp;
    Slice s = slice_of<ES>(p.src, cid, rank);
    bool aborted = false;
#pragma unroll 1
    for (int64_t base = 0; base < n_it; base += 32) {
        // 32 rows' labels at once, and the logits of this warp's rows, a row a lane
        int64_t lab = label0;
        if (base > 0 && p.src.labels && base + lane < n_it) lab = __ldg(p.src.labels + cid + (base + lane) * ncl);
        const bool ok = base + lane < n_it && stream_row_valid(lab, p.src);
        const unsigned valid = __ballot_sync(0xffffffffu, ok);
        float x_lab = 0.f;
        if (p.logp && rank == 0 && ok && (!TOPK || (rp.buf + __popc(valid & lanes_below())) % p.src.buffers == me))
            x_lab = load_scalar<ES>(p.src.x + ((cid + (base + lane) * ncl) * p.src.ld + lab) * ES);
        const int nj = static_cast<int>(min(static_cast<int64_t>(32), n_it - base));
#pragma unroll 1
        for (int j = 0; j < nj; ++j) {
            const int64_t row = cid + (base + j) * ncl;
            if (!(valid >> j & 1u)) {
                if (rank == 0 && me == 0) {
                    if (lane == 0) {
                        if (p.logp) p.logp[row] = 0.f;
                        if (p.entropy) p.entropy[row] = 0.f;
                        if (p.lse) p.lse[row] = 0.f;
                        if (p.stats) p.stats[row] = make_float2(0.f, 0.f);
                    }
                    if (TOPK) {
#pragma unroll 1
                        for (int i = lane; i < p.top_k; i += 32) {
                            p.top_lp[row * p.top_k + i] = 0.f;
                            p.top_ids[row * p.top_k + i] = -1;
                        }
                    }
                }
                continue;
            }
            if (TOPK && rp.buf != me) {
                rp.next(p.src);
                continue;
            }
            const float x_y = __shfl_sync(0xffffffffu, x_lab, j);
            const int buf = rp.buf;
            const uint32_t use = rp.use;
            if (!aborted && !stream_wait(bars, &bars.row_full[buf], use & 1u, p.src.wait_ns)) aborted = true;
            RunStat<ENT, false> st(p.scale);
            stat_collect<kThreads>(st, ex, buf, p.scale);
            if (!TOPK) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.row_empty[buf]);
            }
            int n = 0;
            const int K = p.top_k;
            unsigned long long* best = top[TOPK ? me : 0].list;
            unsigned long long* pushed = reinterpret_cast<unsigned long long*>(smem_pushed);  // the cluster's lists, K each
            if constexpr (TOPK) {  // this CTA's largest, in order
                TopScratch& t = top[me];
                move_slice<ES>(p.src, row, rank, s);
                if (st.s == st.s) n = top_list<ES>(s, maxima + buf * p.max_stride, thread_max[buf], K, t);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.row_empty[buf]);
                top_ordered(best, n);
                if (k > 1) push_list(best, n, K, pushed, rank, k);
            }
            if (k > 1) {
                stat_send(st, ex, k, rank);
                if (!peers_meet(bars, k, aborted ? 0 : p.src.wait_ns)) aborted = true;
                stat_merge(st, ex, k, p.scale);
            }
            st.correct(p.scale);
            const float ln_s = logf(st.s);
            const bool empty = st.s == 0.f;
            if (lane == 0 && rank == 0 && !aborted) {
                if (p.logp) p.logp[row] = empty ? kNegInf : (x_y - st.m) * p.inv_t - ln_s;
                if (ENT) {
                    const float h = ln_s - st.a * kLn2 / st.s;
                    p.entropy[row] = empty || h < 0.f ? 0.f : h;
                }
                if (p.lse) p.lse[row] = empty ? kNegInf : fmaf(st.m, p.inv_t, ln_s);
                if (p.stats) p.stats[row] = make_float2(empty ? kNegInf : st.m, ln_s);
            }
            if constexpr (TOPK) {
                const bool none = !(st.s == st.s);  // a NaN or +inf in the row: no order to speak of
                float* olp = p.top_lp + row * K;
                int32_t* oid = p.top_ids + row * K;
                auto write = [&](int r, unsigned long long item) {
                    if (aborted || none) return;
                    olp[r] = empty ? kNegInf : (float_of_key(static_cast<uint32_t>(item >> 32)) - st.m) * p.inv_t - ln_s;
                    oid[r] = static_cast<int32_t>(~static_cast<uint32_t>(item));
                };
#pragma unroll 1
                for (int i = lane; i < min(n, K); i += 32) {
                    const unsigned long long item = best[i];
                    const int r = k > 1 ? pushed_rank(pushed, K, k, item) : i;
                    if (r < K) write(r, item);
                }
                if (none && rank == 0) {
#pragma unroll 1
                    for (int i = lane; i < K; i += 32) {
                        olp[i] = st.s;
                        oid[i] = -1;
                    }
                }
                __syncwarp();
            }
            rp.next(p.src);
        }
    }
    if (aborted) bars.abort = 1;
}

template <int ES, bool ENT, bool TOPK>
__global__ void __launch_bounds__(kLogprobThreads<TOPK>, 3) logprobs_kernel(const __grid_constant__ LogprobParams p) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ StreamBars bars;
    __shared__ StatExchange ex;
    __shared__ LongSums aside;  // not with top tokens: their rows are one run
    __shared__ TopScratch top[TOPK ? kClosers<TOPK> : 1];
    __shared__ uint32_t thread_max[TOPK ? kClosers<TOPK> : 1][kThreads];  // key of the largest of a thread's blocks, 0: it has none
    using MaxT = typename Block<ES>::type;
    unsigned char* ring = smem;
    MaxT* maxima = reinterpret_cast<MaxT*>(smem + p.src.stages * Sh::kStageBytes);  // of the blocks, max_stride a buffer

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = p.src.k;
    const int rank = k > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int64_t cid = blockIdx.x >> p.src.log2_k, ncl = gridDim.x >> p.src.log2_k;
    const int64_t n_it = stream_rows(p.src, cid);
    stream_init<kThreads>(bars, p.src.stages, k);
    griddep_launch_dependents();  // programmatic dependent launch: no global access before the wait
    griddep_wait();
    // the producer's and closing warps' first 32 rows, the consumers' first one
    const int64_t label0 = first_label(p.src, cid, ncl, warp < Sh::kWarps ? 0 : lane);
    __syncthreads();
    if (k > 1) cluster_arrive_release();  // waited for before the cluster's memory is written to

    if (warp == Sh::kWarps) {
        const bool bad = stream_produce<ES, kThreads>(p.src, bars, ring, 1, cid, ncl, rank, label0);
        // The error word: every CTA adds its labels' bit; the last one publishes and resets.
        if (lane == 0) {
            if (bad) atomicOr(&p.ws->err, static_cast<unsigned>(FOAK_ERRBIT_LABEL_RANGE));
            if (atom_add_acq_rel_gpu(&p.ws->done, 1u) == gridDim.x - 1) {
                const unsigned e = atomicExch(&p.ws->err, 0u);
                if (p.err) *p.err = static_cast<int32_t>(e);
                __threadfence();
                atomicExch(&p.ws->done, 0u);
            }
        }
        __syncwarp();
        if (k > 1) cluster_wait_acquire();
    } else if (warp < Sh::kWarps) {
        StreamPos pos{0, 0, false};
        RowPos rp;
        Slice s = slice_of<ES>(p.src, cid, rank);
        int64_t y_next = label0;
#pragma unroll 1
        for (int64_t it = 0; it < n_it; ++it) {
            const int64_t row = cid + it * ncl;
            const int64_t y = y_next;
            if (p.src.labels && it + 1 < n_it) y_next = __ldg(p.src.labels + row + ncl);
            if (!stream_row_valid(y, p.src)) continue;
            move_slice<ES>(p.src, row, rank, s);
            row_begin(p.src, bars, rp, pos);
            const int buf = rp.buf;
            MaxT* rm = maxima + buf * p.max_stride;
            RunStat<ENT, false> st(p.scale);
            float most = kNegInf;  // of the thread's blocks
            auto chunks = [&](int from, int to) {
#pragma unroll 1
                for (int c0 = from; c0 < to; c0 += Sh::kChunk) {
                    const int nl = min(Sh::kChunk, s.nv - c0);
                    uint4 v[kBlockVec];
                    stream_chunk<kThreads>(p.src, bars, ring, pos, [&](const unsigned char* stage) {
                        if constexpr (TOPK) load_block<ES, kThreads>(stage, nl, v);
                        else load_strided<ES, kThreads>(stage, nl, v);
                    });
                    const float mine = st.template add_vecs<ES>(v, p.scale);
                    if (TOPK) {
                        most = fmaxf(most, mine);
                        const float both = Block<ES>::kPieces > 1 ? fmaxf(mine, __shfl_xor_sync(0xffffffffu, mine, 1)) : mine;
                        if (tid * kBlockVec < nl && tid % Block<ES>::kPieces == 0)
                            rm[kBodyAt + (c0 / kBlockVec + tid) / Block<ES>::kPieces] = static_cast<MaxT>(Block<ES>::pack(both));
                    }
                }
            };
            if constexpr (TOPK) {
                chunks(0, s.nv);
            } else {
#pragma unroll 1
                for (int run = 0; run < s.nv; run += kRunVec<kThreads>) {
                    if (run > 0) {
                        stat_put_aside<ENT, false>(st, aside, run == kRunVec<kThreads>, p.scale);
                        st.restart();
                    }
                    chunks(run, min(s.nv, run + kRunVec<kThreads>));
                }
            }
            if (s.h + s.t > 0 && warp == 0) {  // the head's and the tail's scalars, one a lane
                float e = kNegInf;
                if (tid < s.h + s.t) e = load_scalar<ES>(s.rowp + (tid < s.h ? tid : s.tail_col + (tid - s.h)) * ES);
                st.add(e, p.scale);
                if (TOPK) {
                    const float hm = warp_max_redux(tid < s.h ? e : kNegInf), tm = warp_max_redux(tid < s.h ? kNegInf : e);
                    if (tid == 0) {
                        rm[0] = s.h > 0 ? Block<ES>::pack(hm) : Block<ES>::kNone;
                        rm[1] = s.t > 0 ? Block<ES>::pack(tm) : Block<ES>::kNone;
                    }
                }
            } else if (TOPK && tid == 0) {
                rm[0] = rm[1] = Block<ES>::kNone;
            }
            if (TOPK) thread_max[buf][tid] = tid * kBlockVec < s.nv ? short_key<ES>(most) : 0u;
            if (TOPK || s.nv <= kRunVec<kThreads>) stat_publish(st, ex, buf);
            else stat_publish_long(st, aside, ex, buf, p.scale);
            row_end(bars, buf);
            rp.next(p.src);
        }
        __syncwarp();
        if (k > 1) cluster_wait_acquire();
    } else {
        if (k > 1) cluster_wait_acquire();
        if (!TOPK || warp - (Sh::kWarps + 1) < p.src.buffers)
            close_rows<ES, ENT, TOPK>(p, bars, ex, top, thread_max, maxima,
                                      smem + p.src.stages * Sh::kStageBytes + p.max_bytes, label0);
    }
    __syncthreads();
    if (tid == 0 && stream_aborted(bars) && p.err) {
        // A wait that gave up: its bit follows the word's publication, which is waited for (with a limit).
        const uint64_t t0 = globaltimer_ns();
        while (*reinterpret_cast<volatile unsigned*>(&p.ws->done) != 0 && globaltimer_ns() - t0 < p.src.wait_ns) {
        }
        atomicOr(reinterpret_cast<unsigned*>(p.err), static_cast<unsigned>(FOAK_ERRBIT_TIMEOUT));
    }
    if (k > 1) cluster_sync_converged();  // no CTA leaves while its shared memory may be read
}

template <int ES, bool ENT, bool TOPK>
cudaError_t launch_typed(LogprobParams prm, cudaStream_t stream) {
    auto* kern = &logprobs_kernel<ES, ENT, TOPK>;
    StreamSrc& s = prm.src;
    const int sms = device_sm_count();
    const int64_t nb = s.V * ES / 16 + 1;
    // Two CTAs an SM and slices of 30000 elements for top tokens, whose lists cost a cluster more:
    // with K = 20 rows of 128256 bf16 by 1, 2, 4 and 8 took 19.6, 18.1, 14.5, 14.4 us (1 row),
    // 20.3, 18.9, 15.3, 16.8 (16), 21.8, 23.4, 20.5, 34.9 (64) and 27.3, 26.6, 35.5, 41.5 (130);
    // without 10.5, 8.3, 6.6, 5.8 (1), 11.7, 11.5, 10.2, 13.8 (64), 16.6, 14.8, 16.9, 20.1 (130).
    const int k = cluster_size(s, ES, TOPK ? 30000 : 8 * 1024, 2 * sms);
    set_cluster(s, k);
    const int64_t nblk = (((nb + kBlockVec - 1) / kBlockVec + s.k - 1) / s.k + 1) / Block<ES>::kPieces + 1;
    prm.max_stride = static_cast<int>((kBodyAt + nblk + 63) / 64 * 64);
    const size_t buffer = TOPK ? prm.max_stride * sizeof(typename Block<ES>::type) : 0;
    // As many CTAs an SM as the registers allow (4096 x 32000, K = 5: three 74 us, two 78; K = 0
    // three 48), and a buffer for each closing warp, or fewer
    // of the first, then of the second, where a ring of two stages would not fit.
    const size_t lists = TOPK && s.k > 1 ? static_cast<size_t>(prm.top_k) * s.k * 8 : 0;
    const size_t fixed = 1024 + 256 + sizeof(StreamBars) + sizeof(StatExchange) + lists +
                         (TOPK ? kClosers<TOPK> * (sizeof(TopScratch) + kThreads * 4) : sizeof(LongSums));
    int per_sm = 3;
    // One buffer where every CTA has one row: with three, 320 rows of 128256 fp32 left room for two CTAs
    // an SM, so for two rounds (K = 20: 60 us, 46 with one).
    s.buffers = !TOPK ? 2 : s.N * s.k <= static_cast<int64_t>(sms) * per_sm ? 1 : kClosers<TOPK>;
    auto room_for = [&] { return std::min<int64_t>(228 * 1024 / per_sm, 227 * 1024) - static_cast<int64_t>(fixed + buffer * s.buffers); };
    while (room_for() < 2 * static_cast<int64_t>(Sh::kStageBytes) && (per_sm > 1 || s.buffers > 2)) {
        if (per_sm > 1) {
            --per_sm;
        } else {
            per_sm = 3;
            --s.buffers;
        }
    }
    const int64_t room = room_for();
    if (room < static_cast<int64_t>(Sh::kStageBytes)) return cudaErrorInvalidValue;
    s.stages = static_cast<int>(std::min<size_t>(kStreamMaxStages, room / Sh::kStageBytes));
    prm.max_bytes = static_cast<int>(buffer * s.buffers);
    const size_t smem = static_cast<size_t>(s.stages) * Sh::kStageBytes + prm.max_bytes + lists;
    static SmemLimit limit;
    const cudaError_t e = limit.allow(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    const int64_t clusters = std::max<int64_t>(1, std::min<int64_t>(s.N, static_cast<int64_t>(sms) * per_sm / s.k));
    if (!set_rows(s, clusters)) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * s.k), 1, 1);
    cfg.blockDim = dim3(kLogprobThreads<TOPK>, 1, 1);
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
