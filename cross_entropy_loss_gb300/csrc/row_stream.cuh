// Rows of logits streamed through shared memory by one CTA, or by a cluster of CTAs
// that share a row: the pieces common to the log-probability and distillation kernels.
//
// A CTA has kStreamThreads consumer threads and one producer warp.  The producer
// copies the row in chunks of kStreamChunk 16-byte vectors (one-dimensional bulk
// copies) into a ring of stages; a stage completes on its `full` barrier and is handed
// back by one arrival of every consumer warp on its `empty` barrier.  The producer
// runs ahead of the consumers over the row's end, so the copies of the next row are in
// flight while the consumers finish this one.
//
// Each thread keeps a running (max, sum exp, sum d exp) over the elements it has seen
// (d the exponent), rescaled when a new maximum arrives; the threads' triples meet
// once a row.  Exponents are formed as (x - max) * c, never as x * c - max * c: at
// logits of the type's lowest value the products would overflow and their difference
// would be NaN, and the subtraction is exact where it matters (x near max).
#pragma once

#include <float.h>

#include "common.cuh"
#include "foak_ce.h"
#include "internal.h"
#include "row_common.cuh"

namespace foak {

constexpr int kStreamThreads = 256;                       // consumers
constexpr int kStreamWarps = kStreamThreads / 32;
constexpr int kStreamBlock = kStreamThreads + 32;         // and the producer warp
constexpr int kBlockVec = 4;                              // a thread's vectors of a chunk: one 64-byte block
constexpr int kStreamChunk = kStreamThreads * kBlockVec;  // vectors of a chunk (16 KB)
constexpr uint32_t kStreamStageBytes = kStreamChunk * 16;
constexpr int kStreamMaxStages = 12;
constexpr int kStreamMaxCluster = 8;
constexpr float kMinExp2 = -16384.f;  // 2^x is 0 from far above this; keeps products with it finite

struct StreamSrc {
    const char* x;
    int64_t ld;
    const int64_t* labels;  // null: every row counts and no token is given
    int64_t N, V, ignore_index;
    uint64_t wait_ns;       // limit of every shared-memory barrier wait
    int64_t skip_load_row;  // test hook: this row's first chunk is never loaded (-1: none)
    int k;                  // CTAs of a row's cluster
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
__device__ __forceinline__ void consumers_sync() {
    __syncwarp();
    asm volatile("bar.sync 1, %0;" ::"n"(kStreamThreads) : "memory");
}
// The cluster's barrier, from code whose lanes may have parted.
__device__ __forceinline__ void cluster_sync_converged() {
    __syncwarp();
    cluster_sync();
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
    const int per = ((nb + kBlockVec - 1) / kBlockVec + p.k - 1) / p.k * kBlockVec;
    const int v0 = min(nb, rank * per), v1 = min(nb, v0 + per);
    s.h = rank == 0 ? g.h : 0;
    s.t = rank == p.k - 1 ? g.t : 0;
    s.nv = v1 - v0;
    s.col0 = g.h + static_cast<int64_t>(v0) * EPV;
    s.body = s.rowp + s.col0 * ES;
    s.tail_col = g.h + static_cast<int64_t>(nb) * EPV;
    return s;
}

struct StreamBars {
    uint64_t full[kStreamMaxStages];
    uint64_t empty[kStreamMaxStages];
    int abort;  // a wait gave up: everyone stops waiting and winds down
};

__device__ __forceinline__ void stream_init(StreamBars& b, int stages) {
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&b.full[s], 1);
            mbar_init(&b.empty[s], kStreamWarps);
        }
        b.abort = 0;
        fence_mbar_init();
    }
}

__device__ __forceinline__ bool stream_aborted(const StreamBars& b) { return *reinterpret_cast<const volatile int*>(&b.abort) != 0; }

// Bounded wait that also ends when another thread has given up.
__device__ __forceinline__ bool stream_wait(StreamBars& b, uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
    if (mbar_try_wait(bar, parity)) return true;
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
// row_syncs: cluster barriers the consumers pass in every valid row (0 without a
// cluster); the producer warp takes part in them.
template <int ES>
__device__ __forceinline__ void stream_produce(const StreamSrc& p, StreamBars& bars, unsigned char* ring, int passes,
                                               int64_t cid, int64_t ncl, int rank, int row_syncs) {
    const int lane = threadIdx.x & 31;
    const int64_t n_it = p.N > cid ? (p.N - 1 - cid) / ncl + 1 : 0;
    const uint32_t S = static_cast<uint32_t>(p.stages);
    uint32_t st = 0, par = 0;  // the next stage, and the parity of its use
    bool wrapped = false, stop = false;
    uint32_t armed = 0;  // stages whose last copy was issued
    for (int64_t base = 0; base < n_it; base += 32) {
        // 32 rows' labels at once: no copy waits for a label of its own
        int64_t lab = 0;
        if (p.labels && base + lane < n_it) lab = __ldg(p.labels + cid + (base + lane) * ncl);
        const int nj = static_cast<int>(min(static_cast<int64_t>(32), n_it - base));
        for (int j = 0; j < nj; ++j) {
            const int64_t y = __shfl_sync(0xffffffffu, lab, j);
            if (!stream_row_valid(y, p)) continue;
            const int64_t row = cid + (base + j) * ncl;
            if (lane == 0 && !stop) {
                const Slice s = slice_of<ES>(p, row, rank);
                for (int pass = 0; pass < passes && !stop; ++pass) {
                    for (int c0 = 0; c0 < s.nv; c0 += kStreamChunk) {
                        if (wrapped && !stream_wait(bars, &bars.empty[st], par ^ 1u, p.wait_ns)) stop = true;
                        if (stop || stream_aborted(bars)) {
                            stop = true;
                            break;
                        }
                        if (!(p.skip_load_row == row && pass == 0 && c0 == 0)) {
                            const uint32_t bytes = static_cast<uint32_t>(min(kStreamChunk, s.nv - c0)) * 16u;
                            fence_proxy_async_smem();
                            mbar_arrive_expect_tx(&bars.full[st], bytes);
                            bulk_g2s(ring + st * kStreamStageBytes, s.body + static_cast<int64_t>(c0) * 16, bytes,
                                     &bars.full[st]);
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
            for (int i = 0; i < row_syncs; ++i) cluster_sync();
        }
    }
    // the CTA must not end, nor its shared memory be given away, under a copy in flight
    if (lane == 0) {
        for (uint32_t s = 0; s < S; ++s) {
            if (!(armed >> s & 1u)) continue;
            const uint32_t last = s < st ? par : par ^ 1u;  // the parity of the stage's last use
            (void)mbar_wait_bounded(&bars.full[s], last, p.wait_ns);
        }
    }
    __syncwarp();
}

// A consumer thread's place in the chunk sequence.
struct StreamPos {
    uint32_t st, par;
    bool aborted;
};

// Waits for the next chunk, then read(stage pointer), then hands the stage back.
template <typename F>
__device__ __forceinline__ void stream_chunk(const StreamSrc& p, StreamBars& bars, const unsigned char* ring,
                                             StreamPos& pos, F&& read) {
    if (!pos.aborted && !stream_wait(bars, &bars.full[pos.st], pos.par, p.wait_ns)) pos.aborted = true;
    read(ring + pos.st * kStreamStageBytes);
    __syncwarp();
    if ((threadIdx.x & 31) == 0 && !pos.aborted) mbar_arrive(&bars.empty[pos.st]);
    if (++pos.st == static_cast<uint32_t>(p.stages)) {
        pos.st = 0;
        pos.par ^= 1u;
    }
}

// The thread's block of a chunk: vectors 4 tid .. 4 tid + 3, -inf past the chunk's end.
// They are read in an order turned by tid / 2, so that the eight threads that share a
// 128-byte shared-memory access touch all 32 banks; v is left in that turned order.
template <int ES>
__device__ __forceinline__ void load_block(const unsigned char* stage, int nl, uint4 (&v)[kBlockVec]) {
    const int tid = threadIdx.x;
    const uint4* sb = reinterpret_cast<const uint4*>(stage) + tid * kBlockVec;
#pragma unroll
    for (int i = 0; i < kBlockVec; ++i) {
        const int j = (i + (tid >> 1)) & (kBlockVec - 1);
        v[i] = tid * kBlockVec + j < nl ? sb[j] : RowMath<ES>::pad();
    }
}

// The two floats of pair j of a 16-byte vector's two (fp32) or four (bf16) pairs.
template <int ES>
__device__ __forceinline__ f32x2_t vec_pair(const uint4& v, int j) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (ES == 2) return bf16x2_to_f2(w[j]);
    else return f2_pack(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
}

// Maximum of the vectors' elements; NaN if one of them is.
template <int ES, int NV>
__device__ __forceinline__ float vec_max(const uint4 (&v)[NV]) {
    if constexpr (ES == 2) {
        uint32_t m = bf16x2_max_nan(bf16x2_max_nan(v[0].x, v[0].y), bf16x2_max_nan(v[0].z, v[0].w));
#pragma unroll
        for (int i = 1; i < NV; ++i)
            m = bf16x2_max_nan(m, bf16x2_max_nan(bf16x2_max_nan(v[i].x, v[i].y), bf16x2_max_nan(v[i].z, v[i].w)));
        return max_nan(bf16_lo(m), bf16_hi(m));
    } else {
        float m = kNegInf;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            m = max_nan(m, max_nan(max_nan(__uint_as_float(v[i].x), __uint_as_float(v[i].y)),
                                   max_nan(__uint_as_float(v[i].z), __uint_as_float(v[i].w))));
        return m;
    }
}

// Running softmax statistics of a set of elements: m the maximum (-FLT_MAX while no
// element above -inf was seen), s = sum 2^d, a = sum 2^d d with d = (x - m) c, and
// s2 = sum 2^((x - m) c2) for a second temperature.  NaN and +inf make s NaN.
template <bool ENT, bool TWO>
struct RunStat {
    float m = -FLT_MAX, s = 0.f, a = 0.f, s2 = 0.f;

    __device__ __forceinline__ void raise(float mn, float c, float c2) {
        const float dm = max_nan((m - mn) * c, kMinExp2);
        const float f = ex2(dm);
        if (ENT) a = f * fmaf(dm, s, a);
        s *= f;
        if (TWO) s2 *= ex2(max_nan((m - mn) * c2, kMinExp2));
        m = mn;
    }
    __device__ __forceinline__ void merge(float m2, float sx, float ax, float s2x, float c, float c2) {
        const float mn = max_nan(m, m2);
        raise(mn, c, c2);
        RunStat o;
        o.m = m2;
        o.s = sx;
        o.a = ax;
        o.s2 = s2x;
        o.raise(mn, c, c2);
        s += o.s;
        if (ENT) a += o.a;
        if (TWO) s2 += o.s2;
    }
    __device__ __forceinline__ void add(float x, float c, float c2) {
        if (x == kNegInf) return;
        const float mn = max_nan(m, x);
        if (!(mn == m)) raise(mn, c, c2);
        const float d = max_nan((x - m) * c, kMinExp2);
        const float e = ex2(d);
        s += e;
        if (ENT) a = fmaf(e, d, a);
        if (TWO) s2 += ex2((x - m) * c2);
    }
    // NV vectors whose maximum is bmax
    template <int ES, int NV>
    __device__ __forceinline__ void add_vecs(const uint4 (&v)[NV], float bmax, float c, float c2) {
        if (bmax == kNegInf) return;
        const float mn = max_nan(m, bmax);
        if (!(mn == m)) raise(mn, c, c2);
        const f32x2_t M = f2_pack(-m, -m), C = f2_pack(c, c), C2 = f2_pack(c2, c2);
        f32x2_t ss[2] = {0, 0}, aa[2] = {0, 0}, tt[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int j = 0; j < (ES == 2 ? 4 : 2); ++j) {
                const f32x2_t x = f2_add(vec_pair<ES>(v[i], j), M);
                float lo, hi;
                f2_unpack(f2_mul(x, C), lo, hi);
                if (ENT) {
                    lo = max_nan(lo, kMinExp2);  // 2^-inf * -inf would be NaN
                    hi = max_nan(hi, kMinExp2);
                }
                const f32x2_t e = f2_pack(ex2(lo), ex2(hi));
                ss[j & 1] = f2_add(ss[j & 1], e);
                if (ENT) aa[j & 1] = f2_fma(e, f2_pack(lo, hi), aa[j & 1]);
                if (TWO) tt[j & 1] = f2_add(tt[j & 1], f2_ex2(f2_mul(x, C2)));
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
    }
    // all 32 lanes' sets as one; every lane gets it
    __device__ __forceinline__ void warp_merge(float c, float c2) {
        const float M = warp_max(m);  // drops NaN; the sums below keep it
        raise(M, c, c2);
        s = warp_sum(s);
        if (ENT) a = warp_sum(a);
        if (TWO) s2 = warp_sum(s2);
    }
};

// Shared memory through which the consumers' (and the cluster's) sets meet.
struct StatExchange {
    float4 warp[2][kStreamWarps];           // (m, s, a, s2), by row parity
    float4 cta[2][kStreamMaxCluster];       // the cluster's CTAs' sets, by row parity
};

// Every consumer thread's set as the row's.  One consumer barrier, and with a cluster
// one cluster barrier.
template <bool ENT, bool TWO>
__device__ __forceinline__ void stat_reduce(RunStat<ENT, TWO>& st, StatExchange& ex, uint32_t parity, int k, int rank,
                                            float c, float c2) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    st.warp_merge(c, c2);
    if (lane == 0) ex.warp[parity][warp] = make_float4(st.m, st.s, st.a, st.s2);
    consumers_sync();
    float4 w = ex.warp[parity][lane & (kStreamWarps - 1)];
    st.m = w.x, st.s = w.y, st.a = w.z, st.s2 = w.w;
    float M = st.m;
#pragma unroll
    for (int off = kStreamWarps / 2; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    st.raise(M, c, c2);
#pragma unroll
    for (int off = kStreamWarps / 2; off > 0; off >>= 1) {
        st.s += __shfl_xor_sync(0xffffffffu, st.s, off);
        if (ENT) st.a += __shfl_xor_sync(0xffffffffu, st.a, off);
        if (TWO) st.s2 += __shfl_xor_sync(0xffffffffu, st.s2, off);
    }
    if (k > 1) {
        if (threadIdx.x < static_cast<unsigned>(k)) {
            const uint32_t to = mapa_u32(&ex.cta[parity][rank], threadIdx.x);
            asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(st.m), "f"(st.s), "f"(st.a),
                         "f"(st.s2)
                         : "memory");
        }
        cluster_sync_converged();
        w = ex.cta[parity][0];
        st.m = w.x, st.s = w.y, st.a = w.z, st.s2 = w.w;
        for (int r = 1; r < k; ++r) {
            w = ex.cta[parity][r];
            st.merge(w.x, w.y, w.z, w.w, c, c2);
        }
    }
}

// Number of valid labels, counted by the consumer threads; scratch: kStreamWarps ints.
__device__ __forceinline__ int count_valid_consumers(const StreamSrc& p, int* scratch) {
    if (!p.labels) return static_cast<int>(p.N);
    int cv = 0;
    for (int64_t i0 = threadIdx.x; i0 < p.N; i0 += 8 * kStreamThreads) {
        int64_t y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int64_t i = i0 + static_cast<int64_t>(k) * kStreamThreads;
            y[k] = i < p.N ? __ldg(p.labels + i) : p.ignore_index;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) cv += stream_row_valid(y[k], p);
    }
    cv = __reduce_add_sync(0xffffffffu, cv);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = cv;
    consumers_sync();
    int t = 0;
#pragma unroll
    for (int w = 0; w < kStreamWarps; ++w) t += scratch[w];
    return t;
}

// How a stream kernel is launched: CTAs of a row's cluster, CTAs of an SM, stages.
struct StreamPlan {
    int k, per_sm, stages;
    int64_t grid;
};

}  // namespace foak
