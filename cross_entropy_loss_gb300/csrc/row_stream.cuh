// Rows of logits streamed through shared memory by one CTA, or by a cluster of CTAs
// that share a row: the pieces common to the log-probability and distillation kernels.
//
// A CTA has NT consumer threads (256 or 512), a producer warp and one or more closing
// warps.  The producer copies the row in chunks of 4 NT 16-byte vectors (one-dimensional bulk
// copies) into a ring of stages; a stage completes on its `full` barrier and is handed
// back by one arrival of every consumer warp on its `empty` barrier.  It runs ahead of the
// consumers over the row's end.  The consumers leave each row's partial results in one of
// a few buffers and go on to the next row; a closing warp joins them, with the cluster's
// other CTAs if a row is shared, and does what a row needs once (logarithms, gathers, top
// tokens), so that neither the copies nor the sums wait for it.  That work is a chain of
// latencies: several closing warps take rows in turn.
//
// HBM bounds long rows (8192 x 128256 bf16, sums and entropy: 307 us, 6.85 TB/s, what a copy
// reaches).  Short ones are bounded by issue slots and the ends of rows: 9.2 instructions an
// element and lane group, two thirds of the slots (4096 x 32000: 48 us, 5.4 TB/s).  Two or
// three CTAs an SM hide one's row ends behind another's sums.  The closing warps' code has
// to stay small: unrolled for speed (270 KB of it) it pushed the consumers' own out of the
// instruction cache, 74 against 68 us at K = 5.
//
// Each thread keeps running sums (of 2^d and d 2^d) below a maximum that its warp shares:
// one warp-wide reduction a chunk, and a rescaling only when the warp meets a new maximum
// (rarer and rarer along a row); the warps' sets meet once a row.  The exponent is
// one FMA, d = x c + r with r = -max c rounded once: the sums are then exact for that r,
// and the row's end corrects for its rounding (max c + r, which an FMA gives exactly).
// The rounding of r is an exponent of 64 at most while |max c| < 2^30.  Above that two
// different float32 logits are at least 2^6 apart in the exponent, so an element that is
// not the maximum counts nothing and no exponent is formed.  With two temperatures each
// sum goes by its own scale: at one the logits may be that far apart, at the other not.
#pragma once

#include <float.h>

#include <mutex>

#include "common.cuh"
#include "foak_ce.h"
#include "internal.h"
#include "row_common.cuh"

namespace foak {

constexpr int kBlockVec = 4;  // a thread's vectors of a chunk: one 64-byte block
// What follows from the number of consumer threads.
template <int NT>
struct Shape {
    static constexpr int kWarps = NT / 32;
    static constexpr int kFirstCloser = NT + 32;         // the first closing warp's first thread
    static constexpr int kChunk = NT * kBlockVec;        // vectors of a chunk (16 KB of 256 threads)
    static constexpr uint32_t kStageBytes = kChunk * 16;
};
constexpr int kMaxWarps = 16;
constexpr int kMaxBuffers = 3;                            // rows between the consumers and the closing warps
constexpr int kStreamMaxStages = 12;
constexpr int kStreamMaxCluster = 8;
constexpr float kMinExp2 = -16384.f;  // 2^x is 0 from far above this; keeps products with it finite
constexpr float kFarExp = 1073741824.f;  // 2^30: max c past which two logits differ by an exponent of 64 at least

struct StreamSrc {
    const char* x;
    int64_t ld;
    const int64_t* labels;  // null: every row counts and no token is given
    int64_t N, V, ignore_index;
    uint64_t wait_ns;       // limit of every shared-memory barrier wait
    int64_t skip_load_row;  // test hook: this row's first chunk is never loaded (-1: none)
    int k, log2_k;          // CTAs of a row's cluster
    int64_t each, more;     // rows of every cluster, and how many of the clusters have one more
    int buffers;            // rows between the consumers and the closing warps
    bool evict_last_pass;
    int stages;
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint32_t bf16x2_max_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Barrier of the consumer threads alone (whole warps arrive).
template <int NT>
__device__ __forceinline__ void consumers_sync() {
    __syncwarp();
    asm volatile("bar.sync 1, %0;" ::"n"(NT) : "memory");
}
// Consumers (who do not wait) and closing warps (which do): the number of valid rows is in shared memory.
template <int NT, int CLOSERS>
__device__ __forceinline__ void scale_known() {
    __syncwarp();
    if (threadIdx.x < NT) asm volatile("bar.arrive 2, %0;" ::"n"(NT + 32 * CLOSERS) : "memory");
    else asm volatile("bar.sync 2, %0;" ::"n"(NT + 32 * CLOSERS) : "memory");
}
// The cluster's barrier, from code whose lanes may have parted.
__device__ __forceinline__ void cluster_sync_converged() {
    __syncwarp();
    cluster_sync();
}

// The dynamic shared memory that a kernel has been allowed on each device; it is only ever raised.
// (A fixed array: nothing on the way to a launch allocates, so nothing can throw out of a C entry.)
struct SmemLimit {
    static constexpr int kDevices = 64;
    std::mutex mu;
    size_t allowed[kDevices] = {};

    cudaError_t allow(const void* kern, size_t bytes) {
        int dev = 0;
        const cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
        std::lock_guard<std::mutex> lock(mu);
        if (allowed[dev] >= bytes) return cudaSuccess;
        const cudaError_t set =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
        if (set == cudaSuccess) allowed[dev] = bytes;
        return set;
    }
};

// Launch the work of a cluster size that is a power of two.
inline void set_cluster(StreamSrc& p, int k) {
    p.k = k;
    for (p.log2_k = 0; (1 << p.log2_k) < k;) ++p.log2_k;
}

// The rows shared out to `clusters`: cluster c takes c, c + clusters, ...  False where a
// cluster of several CTAs would get a second row: what its CTAs exchange through is used once.
inline bool set_rows(StreamSrc& p, int64_t clusters) {
    p.each = p.N / clusters;
    p.more = p.N % clusters;
    return p.k == 1 || p.N <= clusters;
}
__device__ __forceinline__ int64_t stream_rows(const StreamSrc& p, int64_t cid) { return p.each + (cid < p.more); }

// How many CTAs share a row: all eight while the rows are few, for a cluster reads its row as
// much faster, and one where there are rows for every SM.  A row of less than kWholeRowBytes
// stays whole, as the exchange costs what the shorter read gains (1 x 32000 bf16: 5.1 us whole,
// 5.4 by two, 5.2 by four or eight; 1 x 128256: 10.5, 8.3, 6.6 and 5.8), and so does a slice of
// less than `least` elements.  `at_most` CTAs run at a time without waiting for one another: a
// shared row is its cluster's only one.
constexpr int64_t kWholeRowBytes = 96 * 1024;
inline int cluster_size(const StreamSrc& p, int es, int64_t least, int64_t at_most) {
    if (p.V * es < kWholeRowBytes) return 1;
    int k = kStreamMaxCluster;
    while (k > 1 && (p.N * k > at_most || p.V < k * least)) k /= 2;
    return k;
}

__device__ __forceinline__ bool stream_row_valid(int64_t y, const StreamSrc& p) {
    return !p.labels || (y != p.ignore_index && y >= 0 && y < p.V);
}

// A CTA's share of a row: whole 64-byte blocks of the aligned body; the scalars before
// the first 16-byte boundary go to the first CTA, those after the last to the last one.
struct Slice {
    const char* rowp;
    const char* body;  // the slice's first vector
    int h, t;          // scalars of the head and tail, if they are this CTA's
    int nv;            // vectors of the slice
    int64_t col0;      // column of the slice's first vector
    int64_t tail_col;
};

template <int ES>
__device__ __forceinline__ Slice slice_of(const StreamSrc& p, int64_t row, int rank) {
    constexpr int EPV = 16 / ES;
    Slice s;
    s.rowp = p.x + row * p.ld * ES;
    const RowGeom g = row_geom<ES>(s.rowp, p.V);
    const int nb = static_cast<int>(g.nb);
    const int per = (((nb + kBlockVec - 1) / kBlockVec + p.k - 1) >> p.log2_k) * kBlockVec;
    const int v0 = min(nb, rank * per), v1 = min(nb, v0 + per);
    s.h = rank == 0 ? g.h : 0;
    s.t = rank == p.k - 1 ? g.t : 0;
    s.nv = v1 - v0;
    s.col0 = g.h + static_cast<int64_t>(v0) * EPV;
    s.body = s.rowp + s.col0 * ES;
    s.tail_col = g.h + static_cast<int64_t>(nb) * EPV;
    return s;
}
// The slice of another row, from one whose row starts at the same offset modulo 16 bytes
// (every row does when the row stride is a multiple of 16 bytes).
template <int ES>
__device__ __forceinline__ void move_slice(const StreamSrc& p, int64_t row, int rank, Slice& s) {
    if ((p.ld * ES & 15) == 0) {
        s.rowp = p.x + row * p.ld * ES;
        s.body = s.rowp + s.col0 * ES;
    } else {
        s = slice_of<ES>(p, row, rank);
    }
}

struct StreamBars {
    uint64_t full[kStreamMaxStages];
    uint64_t empty[kStreamMaxStages];
    uint64_t row_full[kMaxBuffers];    // the consumers' part of a row is in its buffer: one arrival a consumer warp
    uint64_t row_empty[kMaxBuffers];   // the closing warp has taken it
    uint64_t row_ready[kMaxBuffers];   // the closing warp has what the second sweep needs
    uint64_t row_stored[kMaxBuffers];  // the second sweep's stores are made: one arrival a consumer warp
    uint64_t peers;                    // the cluster's CTAs have sent their part of its row: one arrival a CTA
    int abort;              // a wait gave up: everyone stops waiting and winds down
};

template <int NT>
__device__ __forceinline__ void stream_init(StreamBars& b, int stages, int cluster) {
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&b.full[s], 1);
            mbar_init(&b.empty[s], Shape<NT>::kWarps);
        }
        for (int i = 0; i < kMaxBuffers; ++i) {
            mbar_init(&b.row_full[i], Shape<NT>::kWarps);
            mbar_init(&b.row_empty[i], 1);
            mbar_init(&b.row_ready[i], 1);
            mbar_init(&b.row_stored[i], Shape<NT>::kWarps);
        }
        mbar_init(&b.peers, cluster);
        b.abort = 0;
        fence_mbar_init();
    }
}

__device__ __forceinline__ bool stream_aborted(const StreamBars& b) { return *reinterpret_cast<const volatile int*>(&b.abort) != 0; }

// Bounded wait that also ends when another thread has given up.
__device__ __forceinline__ bool stream_wait(StreamBars& b, uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
    if (__builtin_expect(mbar_try_wait(bar, parity), 1)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 255u) == 0) {
            if (stream_aborted(b)) return false;
            if (globaltimer_ns() - t0 > limit_ns) {
                b.abort = 1;
                return false;
            }
        }
    }
}

// The producer warp: rows cid, cid + ncl, ...; every valid row's chunks `passes` times.
// first: the label of the lane's first row (the first 32 rows are loaded ahead).  Returns
// whether a label was bad.
template <int ES, int NT>
__device__ __forceinline__ bool stream_produce(const StreamSrc& p, StreamBars& bars, unsigned char* ring, int passes,
                                               int64_t cid, int64_t ncl, int rank, int64_t first) {
    const int lane = threadIdx.x & 31;
    const int64_t n_it = stream_rows(p, cid);
    const uint32_t S = static_cast<uint32_t>(p.stages);
    Slice s = slice_of<ES>(p, cid, rank);
    uint32_t st = 0, par = 0;  // the next stage, and the parity of its use
    bool wrapped = false, stop = false;
    uint32_t armed = 0;  // stages whose last copy was issued
    bool bad = false;
#pragma unroll 1
    for (int64_t base = 0; base < n_it; base += 32) {
        // 32 rows' labels at once: no copy waits for a label of its own
        int64_t lab = first;
        if (base > 0 && p.labels && base + lane < n_it) lab = __ldg(p.labels + cid + (base + lane) * ncl);
        const bool ok = base + lane < n_it && stream_row_valid(lab, p);
        bad |= base + lane < n_it && !ok && lab != p.ignore_index;
        const unsigned valid = __ballot_sync(0xffffffffu, ok);
        const int nj = static_cast<int>(min(static_cast<int64_t>(32), n_it - base));
#pragma unroll 1
        for (int j = 0; j < nj; ++j) {
            if (!(valid >> j & 1u)) continue;
            const int64_t row = cid + (base + j) * ncl;
            if (lane == 0 && !stop) {
                move_slice<ES>(p, row, rank, s);
#pragma unroll 1
                for (int pass = 0; pass < passes && !stop; ++pass) {
#pragma unroll 1
                    for (int c0 = 0; c0 < s.nv; c0 += Shape<NT>::kChunk) {
                        if (wrapped && !stream_wait(bars, &bars.empty[st], par ^ 1u, p.wait_ns)) stop = true;
                        if (stop || stream_aborted(bars)) {
                            stop = true;
                            break;
                        }
                        if (!(p.skip_load_row == row && pass == 0 && c0 == 0)) {
                            const uint32_t bytes = static_cast<uint32_t>(min(Shape<NT>::kChunk, s.nv - c0)) * 16u;
                            fence_proxy_async_smem();
                            mbar_arrive_expect_tx(&bars.full[st], bytes);
                            const char* from = s.body + static_cast<int64_t>(c0) * 16;
                            // the last sweep's reads let the row go from L2, where the rows between two sweeps wait
                            if (p.evict_last_pass && pass == passes - 1)
                                bulk_g2s_hint(ring + st * Shape<NT>::kStageBytes, from, bytes, &bars.full[st],
                                              l2_policy_evict_first());
                            else
                                bulk_g2s(ring + st * Shape<NT>::kStageBytes, from, bytes, &bars.full[st]);
                            armed |= 1u << st;
                        } else {
                            armed &= ~(1u << st);
                        }
                        if (++st == S) {
                            st = 0;
                            par ^= 1u;
                            wrapped = true;
                        }
                    }
                }
            }
            __syncwarp();
        }
    }
    // the CTA must not end, nor its shared memory be given away, under a copy in flight
    if (lane == 0) {
#pragma unroll 1
        for (uint32_t s = 0; s < S; ++s) {
            if (!(armed >> s & 1u)) continue;
            const uint32_t last = s < st ? par : par ^ 1u;  // the parity of the stage's last use
            (void)mbar_wait_bounded(&bars.full[s], last, p.wait_ns);
        }
    }
    return __any_sync(0xffffffffu, bad);
}
// The label of a lane's or thread's first row.
__device__ __forceinline__ int64_t first_label(const StreamSrc& p, int64_t cid, int64_t ncl, int it) {
    const int64_t row = cid + it * ncl;
    return p.labels && row < p.N ? __ldg(p.labels + row) : 0;
}

// A consumer thread's place in the chunk sequence.
struct StreamPos {
    uint32_t st, par;
    bool aborted;
};

// Waits for the next chunk, then read(stage pointer), then hands the stage back.
template <int NT, typename F>
__device__ __forceinline__ void stream_chunk(const StreamSrc& p, StreamBars& bars, const unsigned char* ring,
                                             StreamPos& pos, F&& read) {
    if (!pos.aborted && !stream_wait(bars, &bars.full[pos.st], pos.par, p.wait_ns)) pos.aborted = true;
    read(ring + pos.st * Shape<NT>::kStageBytes);
    __syncwarp();
    if ((threadIdx.x & 31) == 0 && !pos.aborted) mbar_arrive(&bars.empty[pos.st]);
    if (++pos.st == static_cast<uint32_t>(p.stages)) {
        pos.st = 0;
        pos.par ^= 1u;
    }
}

// A valid row's place in the exchange between the consumers and the closing warps.
struct RowPos {
    uint32_t n = 0;    // valid rows so far
    int buf = 0;       // the buffer
    uint32_t use = 0;  // and which use of it
    __device__ __forceinline__ void next(const StreamSrc& p) {
        ++n;
        if (++buf == p.buffers) {
            buf = 0;
            ++use;
        }
    }
};
// Consumers, before they write into the row's buffer: its last use is taken.
__device__ __forceinline__ void row_begin(const StreamSrc& p, StreamBars& bars, const RowPos& row, StreamPos& pos) {
    if (row.use > 0 && !pos.aborted && !stream_wait(bars, &bars.row_empty[row.buf], (row.use & 1u) ^ 1u, p.wait_ns))
        pos.aborted = true;
}
// Consumers: the warp's part of the row is written.
__device__ __forceinline__ void row_end(StreamBars& bars, int buf) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bars.row_full[buf]);
}

// One arrival on the barrier `bar` of another CTA of the cluster, releasing this thread's writes to it.
__device__ __forceinline__ void remote_arrive(uint64_t* bar, uint32_t rank) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(mapa_u32(bar, rank)) : "memory");
}
// Bounded wait for the cluster's arrivals, acquiring what they released.
__device__ __forceinline__ bool peers_wait(StreamBars& b, uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 1;; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((i & 255u) == 0) {
            if (stream_aborted(b)) return false;
            if (globaltimer_ns() - t0 > limit_ns) {
                b.abort = 1;
                return false;
            }
        }
    }
}

// The thread's block of a chunk: vectors 4 tid .. 4 tid + 3, -inf past the chunk's end.
// They are read in an order turned by tid / 2, so that the eight threads that share a
// 128-byte shared-memory access touch all 32 banks; v is left in that turned order.
template <int ES, int NT>
__device__ __forceinline__ void load_block(const unsigned char* stage, int nl, uint4 (&v)[kBlockVec]) {
    const int tid = threadIdx.x, turn = tid >> 1 & (kBlockVec - 1);
    const uint4* sb = reinterpret_cast<const uint4*>(stage) + tid * kBlockVec;
    if (nl == Shape<NT>::kChunk) {
#pragma unroll
        for (int i = 0; i < kBlockVec; ++i) v[i] = sb[i ^ turn];
    } else {
#pragma unroll
        for (int i = 0; i < kBlockVec; ++i) v[i] = tid * kBlockVec + (i ^ turn) < nl ? sb[i ^ turn] : RowMath<ES>::pad();
    }
}
// Four vectors of a chunk without a block's order: tid, tid + NT, ...
template <int ES, int NT>
__device__ __forceinline__ void load_strided(const unsigned char* stage, int nl, uint4 (&v)[kBlockVec]) {
    const int tid = threadIdx.x;
    const uint4* sb = reinterpret_cast<const uint4*>(stage) + tid;
    if (nl == Shape<NT>::kChunk) {
#pragma unroll
        for (int i = 0; i < kBlockVec; ++i) v[i] = sb[i * NT];
    } else {
#pragma unroll
        for (int i = 0; i < kBlockVec; ++i)
            v[i] = tid + i * NT < nl ? sb[i * NT] : RowMath<ES>::pad();
    }
}

// The two floats of pair j of a 16-byte vector's two (fp32) or four (bf16) pairs.
template <int ES>
__device__ __forceinline__ f32x2_t vec_pair(const uint4& v, int j) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (ES == 2) return bf16x2_to_f2(w[j]);
    else return f2_pack(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
}

// Scales of the exponents: c = log2(e) / T, a second one for a second temperature, and the
// value below which a logit's exponential is 0 whatever the maximum (see RunStat::far).
struct ExpScale {
    float c, c2, low;
};
__host__ __device__ __forceinline__ ExpScale exp_scale(float temperature) {
    ExpScale s;
    s.c = kLog2e / temperature;
    s.c2 = kLog2e;
    s.low = -4.f * kFarExp / s.c;
    return s;
}

// Running softmax statistics.  m is the warp's maximum (-FLT_MAX while no element above
// -inf was seen), s = sum 2^d, a = sum 2^d d the thread's sums, with d = x c + r, r = -m c,
// and s2 = sum 2^(x c2 + r2) for a second temperature.  NaN and +inf make s NaN.
template <bool ENT, bool TWO>
struct RunStat {
    float m = -FLT_MAX, r, r2, s = 0.f, a = 0.f, s2 = 0.f;

    __device__ __forceinline__ explicit RunStat(const ExpScale& x) : r(FLT_MAX * x.c), r2(FLT_MAX * x.c2) {}

    // one of the scales is far (each sum goes by its own)
    __device__ __forceinline__ bool far(const ExpScale& x) const { return far(m, x.c) || (TWO && far(m, x.c2)); }
    static __device__ __forceinline__ bool far(float m, float c) { return fabsf(m) * c >= kFarExp && fabsf(m) <= FLT_MAX; }

    // r has to be this rounded product wherever it is used: not to be contracted into an FMA
    static __device__ __forceinline__ float minus_product(float m, float c) { return __fmul_rn(-m, c); }

    // The same sums below a maximum mn >= m (fmaxf also turns a NaN into 2^-16384 = 0: it is in the sums).
    __device__ __forceinline__ void raise(float mn, const ExpScale& x) {
        const float rn = minus_product(mn, x.c);
        const float dm = mn == m ? 0.f : far(mn, x.c) ? kMinExp2 : fmaxf(rn - r, kMinExp2);
        const float f = ex2(dm);
        if (ENT) a = f * fmaf(dm, s, a);
        s *= f;
        if (TWO) {
            const float rn2 = minus_product(mn, x.c2);
            s2 *= mn == m ? 1.f : far(mn, x.c2) ? 0.f : ex2(fmaxf(rn2 - r2, kMinExp2));
            r2 = rn2;
        }
        m = mn;
        r = rn;
    }
    __device__ __forceinline__ void set(const float4& w, const ExpScale& x) {
        m = w.x, s = w.y, a = w.z, s2 = w.w;
        r = minus_product(m, x.c);
        if (TWO) r2 = minus_product(m, x.c2);
    }
    // Sums of 0 below the same maximum.
    __device__ __forceinline__ void restart() { s = a = s2 = 0.f; }
    // One element a lane (-inf: none), by the whole warp.
    __device__ __forceinline__ void add(float v, const ExpScale& x) {
        const float mn = fmaxf(m, warp_max_redux(v));
        if (mn > m) raise(mn, x);
        if (v == kNegInf) return;
        if (__builtin_expect(far(x), 0)) {
            add_far(v, far(m, x.c), TWO && far(m, x.c2), x);
            return;
        }
        const float d = max_nan(fmaf(v, x.c, r), kMinExp2);
        const float e = ex2(d);
        s += e;
        if (ENT) a = fmaf(e, d, a);
        if (TWO) s2 += ex2(fmaf(v, x.c2, r2));
    }
    // NV vectors a lane, by the whole warp; returns the maximum of the lane's (NaN aside).
    template <int ES, int NV>
    __device__ __forceinline__ float add_vecs(const uint4 (&v)[NV], const ExpScale& x) {
        const float bmax = RowMath<ES>::template vmax<NV>(v);
        const float mn = fmaxf(m, warp_max_redux(bmax));
        if (mn > m) raise(mn, x);
        if (__builtin_expect(far(x), 0)) {
            add_vecs_far<ES, NV>(v, x);
            return bmax;
        }
        const f32x2_t C = f2_pack(x.c, x.c), R = f2_pack(r, r), C2 = f2_pack(x.c2, x.c2), R2 = f2_pack(r2, r2);
        f32x2_t ss[2] = {0, 0}, aa[2] = {0, 0}, tt[2] = {0, 0};
        const uint32_t low2 = pack_bf16x2(x.low, x.low);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            uint4 w = v[i];
            // -inf, and what is as far below, to where 2^d is 0 and d finite: 0 * -inf would be NaN
            if (ENT && ES == 2) {
                w.x = bf16x2_max_nan(w.x, low2), w.y = bf16x2_max_nan(w.y, low2);
                w.z = bf16x2_max_nan(w.z, low2), w.w = bf16x2_max_nan(w.w, low2);
            }
            if (ENT && ES == 4) {
                w.x = __float_as_uint(max_nan(__uint_as_float(w.x), x.low));
                w.y = __float_as_uint(max_nan(__uint_as_float(w.y), x.low));
                w.z = __float_as_uint(max_nan(__uint_as_float(w.z), x.low));
                w.w = __float_as_uint(max_nan(__uint_as_float(w.w), x.low));
            }
#pragma unroll
            for (int j = 0; j < (ES == 2 ? 4 : 2); ++j) {
                const f32x2_t e = vec_pair<ES>(w, j);
                const f32x2_t d = f2_fma(e, C, R);
                const f32x2_t p = f2_ex2(d);
                ss[j & 1] = f2_add(ss[j & 1], p);
                if (ENT) aa[j & 1] = f2_fma(p, d, aa[j & 1]);
                if (TWO) tt[j & 1] = f2_add(tt[j & 1], f2_ex2(f2_fma(e, C2, R2)));
            }
        }
        float lo, hi;
        f2_unpack(f2_add(ss[0], ss[1]), lo, hi);
        s += lo + hi;
        if (ENT) {
            f2_unpack(f2_add(aa[0], aa[1]), lo, hi);
            a += lo + hi;
        }
        if (TWO) {
            f2_unpack(f2_add(tt[0], tt[1]), lo, hi);
            s2 += lo + hi;
        }
        return bmax;
    }
    // An element's term where its scale is far (1 if it is the maximum) or not.
    __device__ __forceinline__ float term(float v, bool is_far, float c, float rc) const {
        if (is_far) return v == m ? 1.f : v == v ? 0.f : v;
        return ex2(max_nan(fmaf(v, c, rc), kMinExp2));
    }
    // An element where a scale is far: the entropy, which goes with the first, gets nothing
    // from an element at the maximum.
    __device__ __forceinline__ void add_far(float v, bool one, bool two, const ExpScale& x) {
        static_assert(!(ENT && TWO), "a first scale that is not far would need its part of the entropy");
        s += term(v, !TWO || one, x.c, r);
        if (TWO) s2 += term(v, two, x.c2, r2);
    }
    template <int ES, int NV>
    __device__ __forceinline__ void add_vecs_far(const uint4 (&v)[NV], const ExpScale& x) {
        const bool one = far(m, x.c), two = TWO && far(m, x.c2);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int j = 0; j < (ES == 2 ? 4 : 2); ++j) {
                float lo, hi;
                f2_unpack(vec_pair<ES>(v[i], j), lo, hi);
                add_far(lo, one, two, x);
                add_far(hi, one, two, x);
            }
        }
    }
    // The sums as those of exponents (x - m) c, for an r that is m c exactly.
    __device__ __forceinline__ void correct(const ExpScale& x) {
        if (!far(m, x.c)) {
            const float e = fmaf(m, x.c, r), f = ex2(-e);
            if (ENT) a = f * fmaf(-e, s, a);
            s *= f;
        }
        if (TWO && !far(m, x.c2)) s2 *= ex2(-fmaf(m, x.c2, r2));
    }
};

// Shared memory through which the consumers' (and the cluster's) sets meet.
struct StatExchange {
    float4 warp[kMaxBuffers][kMaxWarps];  // (m, s, a, s2), by row buffer
    float4 cta[kStreamMaxCluster];        // the cluster's CTAs' sets of its row
};

// The sums of a long row's earlier runs of kRunChunks chunks, by consumer warp: each as two
// floats (a sum and what its additions lost), below the maximum m.  A thread adds once a chunk, and
// a chain of float additions of equal numbers rounds the same way for long: without the
// runs, 134 million fp32 logits of two values (4096 chunks a CTA) left ln S off by 3.2e-5, 2^31
// bf16 ones by 9.5e-5.
constexpr int kRunChunks = 64;
struct LongSums {
    float m[kMaxWarps];
    float2 s[kMaxWarps], a[kMaxWarps], s2[kMaxWarps];
};
template <int NT>
constexpr int kRunVec = kRunChunks * Shape<NT>::kChunk;  // a run's vectors

// x + y = sum + error exactly
__device__ __forceinline__ void add_exactly(float2& x, float y) {
    const float sum = __fadd_rn(x.x, y), b = __fsub_rn(sum, x.x);
    x.y += __fadd_rn(__fsub_rn(x.x, __fsub_rn(sum, b)), __fsub_rn(y, b));
    x.x = sum;
}
// The warp's sums since the last time put with the earlier ones (out of line: few rows are so long).
template <bool ENT, bool TWO>
__device__ __noinline__ void stat_put_aside(RunStat<ENT, TWO> st, LongSums& l, bool first, const ExpScale x) {
    const int warp = threadIdx.x >> 5;
    st.s = warp_sum(st.s);
    if (ENT) st.a = warp_sum(st.a);
    if (TWO) st.s2 = warp_sum(st.s2);
    if ((threadIdx.x & 31) == 0) {
        RunStat<ENT, TWO> sum(x), lost(x);
        if (!first) {
            sum.set(make_float4(l.m[warp], l.s[warp].x, l.a[warp].x, l.s2[warp].x), x);
            lost.set(make_float4(l.m[warp], l.s[warp].y, l.a[warp].y, l.s2[warp].y), x);
        }
        sum.raise(st.m, x);
        lost.raise(st.m, x);
        l.m[warp] = st.m;
        float2 t = make_float2(sum.s, lost.s);
        add_exactly(t, st.s);
        l.s[warp] = t;
        t = make_float2(sum.a, lost.a);
        if (ENT) add_exactly(t, st.a);
        l.a[warp] = t;
        t = make_float2(sum.s2, lost.s2);
        if (TWO) add_exactly(t, st.s2);
        l.s2[warp] = t;
    }
    __syncwarp();
}

// Every warp's set put into the exchange; a consumer barrier has to follow.
template <bool ENT, bool TWO>
__device__ __forceinline__ void stat_publish(RunStat<ENT, TWO>& st, StatExchange& ex, int buf) {
    st.s = warp_sum(st.s);
    if (ENT) st.a = warp_sum(st.a);
    if (TWO) st.s2 = warp_sum(st.s2);
    if ((threadIdx.x & 31) == 0) ex.warp[buf][threadIdx.x >> 5] = make_float4(st.m, st.s, st.a, st.s2);
}
// The same of a row of several runs, whose last one is in st.
template <bool ENT, bool TWO>
__device__ __forceinline__ void stat_publish_long(const RunStat<ENT, TWO>& st, LongSums& l, StatExchange& ex, int buf,
                                                  const ExpScale& x) {
    stat_put_aside<ENT, TWO>(st, l, false, x);
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0)
        ex.warp[buf][warp] = make_float4(l.m[warp], l.s[warp].x + l.s[warp].y, l.a[warp].x + l.a[warp].y,
                                         l.s2[warp].x + l.s2[warp].y);
}
// The CTA's set from its warps', by whole warps; every lane gets it.
template <int NT, bool ENT, bool TWO>
__device__ __forceinline__ void stat_collect(RunStat<ENT, TWO>& st, const StatExchange& ex, int buf,
                                             const ExpScale& x) {
    st.set(ex.warp[buf][threadIdx.x & (Shape<NT>::kWarps - 1)], x);
    st.raise(warp_max_redux(st.m), x);
#pragma unroll
    for (int off = Shape<NT>::kWarps / 2; off > 0; off >>= 1) {
        st.s += __shfl_xor_sync(0xffffffffu, st.s, off);
        if (ENT) st.a += __shfl_xor_sync(0xffffffffu, st.a, off);
        if (TWO) st.s2 += __shfl_xor_sync(0xffffffffu, st.s2, off);
    }
}
// In a cluster, by the closing warps of its row: this CTA's set to every CTA, then, when all
// have met, the row's from all.
__device__ __forceinline__ bool peers_meet(StreamBars& bars, int k, uint64_t limit_ns) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
    if (lane < k) remote_arrive(&bars.peers, static_cast<uint32_t>(lane));
    __syncwarp();
    return peers_wait(bars, &bars.peers, 0, limit_ns);
}
template <bool ENT, bool TWO>
__device__ __forceinline__ void stat_send(const RunStat<ENT, TWO>& st, StatExchange& ex, int k, int rank) {
    const int lane = threadIdx.x & 31;
    if (lane < k) {
        const uint32_t to = mapa_u32(&ex.cta[rank], static_cast<uint32_t>(lane));
        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(st.m), "f"(st.s), "f"(st.a),
                     "f"(st.s2)
                     : "memory");
    }
}
template <bool ENT, bool TWO>
__device__ __forceinline__ void stat_merge(RunStat<ENT, TWO>& st, const StatExchange& ex, int k, const ExpScale& x) {
    st.set(ex.cta[threadIdx.x & (k - 1)], x);
    st.raise(warp_max_redux(st.m), x);
#pragma unroll 1
    for (int off = k / 2; off > 0; off >>= 1) {
        st.s += __shfl_xor_sync(0xffffffffu, st.s, off);
        if (ENT) st.a += __shfl_xor_sync(0xffffffffu, st.a, off);
        if (TWO) st.s2 += __shfl_xor_sync(0xffffffffu, st.s2, off);
    }
}

// Number of valid labels, counted by the consumer threads; scratch: an int a warp.
template <int NT>
__device__ __forceinline__ int count_valid_consumers(const StreamSrc& p, int* scratch) {
    if (!p.labels) return static_cast<int>(p.N);
    int cv = 0;
    for (int64_t i0 = threadIdx.x; i0 < p.N; i0 += 8 * NT) {
        int64_t y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int64_t i = i0 + static_cast<int64_t>(k) * NT;
            y[k] = i < p.N ? __ldg(p.labels + i) : p.ignore_index;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) cv += stream_row_valid(y[k], p);
    }
    cv = __reduce_add_sync(0xffffffffu, cv);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = cv;
    consumers_sync<NT>();
    int t = 0;
#pragma unroll
    for (int w = 0; w < Shape<NT>::kWarps; ++w) t += scratch[w];
    return t;
}

}  // namespace foak
