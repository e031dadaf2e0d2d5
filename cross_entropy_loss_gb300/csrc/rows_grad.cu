// Backward passes from saved row statistics: the gradient of log probabilities and
// entropies (logprobs.cu), and of the distillation loss (distill.cu).  With the
// statistics known every element is independent, so this is a stream over (row, 32 KB
// segment) work items, 256 threads each, eight 16-byte loads in flight per thread
// before the arithmetic.  Rows that do not count are only written (+0.0).
//
//   log probabilities, entropy (d = (x - m) / T - ln S = ln p):
//     dx_j = ([j = y] - p_j) g_l / T - p_j (d_j + H) g_h / T = p_j (A + B d_j) + [j = y] g_l / T
//   distillation: a1 e^{x_j - m} + aT e^{(x_j - m) / T}, and the label's and the teacher's
//     tokens rewritten after a barrier, from logits read before it (the gradient may
//     replace the logits).
//
// The statistics are (m, ln S), not their sum: at |m| past 2^24 ln n the sum has lost
// ln S, and a row of n equal lowest values would get p = 1 instead of 1 / n.
//
// HBM bounds both.  Log probabilities and entropy: 8192 x 128256 bf16 670 us (6.3 TB/s read and
// written), 4096 x 32000 87 us (6.0).  Distillation, K = 128: 8192 x 128256
// 725 us (5.8 TB/s), 4096 x 32000, K = 64: 91 us, and 1 to 3 us for clearing its error word.  No
// ring here: a thread's own 128 bytes in flight times 1024 threads an SM are twice what covers
// the latency, and nothing is read twice.
#include <algorithm>

#include "common.cuh"
#include "foak_ce.h"
#include "internal.h"
#include "row_stream.cuh"
#include "teacher.cuh"

namespace foak {

namespace {

constexpr int kGradThreads = 256;
constexpr int kGradVpt = 8;
constexpr int kGradSegVec = kGradThreads * kGradVpt;  // 32 KB
constexpr int kGradBlocksPerSm = 4;
constexpr int kTeacherBlocksPerSm = 3;  // 8192 x 128256 bf16, K = 128: 718 us, by four 742 (at three 24-60 bytes spill)

struct RowsGradParams {
    StreamSrc src;
    char* dx;
    int64_t nseg;
    float inv_t, c;
    int32_t* err;
    // log probabilities and entropy
    const float2* stats2;
    const float* entropy;
    const float* grad_logp;     // null: 0
    const float* grad_entropy;  // null: 0
    // distillation
    const float4* stats4;
    TeacherSrc teacher;
    const float* g_ptr;  // null: 1
    float denom, ce_w, kd_w;
};

// One segment of a row: its vectors, and the row's scalars if they are its.
struct Segment {
    int64_t row;
    const char* rowp;
    char* drow;
    int vbeg, vend;   // vectors of the row's body
    int h;            // the row's head scalars
    int n_edge;       // head and tail scalars of this segment
    int64_t col_lo, col_hi, tail_col;
    bool first;
};

template <int ES>
__device__ __forceinline__ Segment segment_of(const RowsGradParams& p, int64_t item) {
    constexpr int EPV = 16 / ES;
    Segment s;
    s.row = item / p.nseg;
    const int seg = static_cast<int>(item - s.row * p.nseg);
    s.rowp = p.src.x + s.row * p.src.ld * ES;
    s.drow = p.dx + s.row * p.src.ld * ES;
    const RowGeom g = row_geom<ES>(s.rowp, p.src.V);
    const int nb = static_cast<int>(g.nb);
    s.first = seg == 0;
    const bool last = seg == p.nseg - 1;
    s.vbeg = min(nb, seg * kGradSegVec);
    s.vend = last ? nb : min(nb, s.vbeg + kGradSegVec);
    s.h = g.h;
    s.tail_col = g.h + static_cast<int64_t>(nb) * EPV;
    s.n_edge = (s.first ? g.h : 0) + (last ? g.t : 0);
    s.col_lo = s.first ? 0 : g.h + static_cast<int64_t>(s.vbeg) * EPV;
    s.col_hi = last ? p.src.V : g.h + static_cast<int64_t>(s.vend) * EPV;
    return s;
}

__device__ __forceinline__ int64_t edge_column(const Segment& s, int i) {
    const int h = s.first ? s.h : 0;
    return i < h ? i : s.tail_col + (i - h);
}

template <int ES>
__device__ __forceinline__ void zero_segment(const Segment& s) {
    uint4* dst = reinterpret_cast<uint4*>(s.drow + static_cast<int64_t>(s.h) * ES);
    for (int v = s.vbeg + threadIdx.x; v < s.vend; v += kGradThreads) st_global_cs_v4(dst + v, make_uint4(0u, 0u, 0u, 0u));
    if (static_cast<int>(threadIdx.x) < s.n_edge) store_scalar<ES>(s.drow + edge_column(s, threadIdx.x) * ES, 0.f);
}

template <int ES>
__device__ __forceinline__ void load_segment(const Segment& s, uint4 (&v)[kGradVpt], float& edge) {
    const uint4* src = reinterpret_cast<const uint4*>(s.rowp + static_cast<int64_t>(s.h) * ES);
#pragma unroll
    for (int i = 0; i < kGradVpt; ++i) {
        const int vv = s.vbeg + threadIdx.x + i * kGradThreads;
        v[i] = RowMath<ES>::pad();
        if (vv < s.vend) v[i] = ld_global_v4(src + vv);
    }
    edge = 0.f;
    if (static_cast<int>(threadIdx.x) < s.n_edge) edge = load_scalar<ES>(s.rowp + edge_column(s, threadIdx.x) * ES);
}

// f maps a pair of logits to the pair of their gradients
template <int ES, typename F>
__device__ __forceinline__ void store_segment(const Segment& s, const uint4 (&v)[kGradVpt], float edge, F&& f) {
    uint4* dst = reinterpret_cast<uint4*>(s.drow + static_cast<int64_t>(s.h) * ES);
#pragma unroll
    for (int i = 0; i < kGradVpt; ++i) {
        const int vv = s.vbeg + threadIdx.x + i * kGradThreads;
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < (ES == 2 ? 4 : 2); ++j) {
            const f32x2_t e = f(vec_pair<ES>(v[i], j));
            if constexpr (ES == 2) {
                o[j] = f2_to_bf16x2(e);
            } else {
                float lo, hi;
                f2_unpack(e, lo, hi);
                o[2 * j] = __float_as_uint(lo);
                o[2 * j + 1] = __float_as_uint(hi);
            }
        }
        if (vv < s.vend) st_global_cs_v4(dst + vv, make_uint4(o[0], o[1], o[2], o[3]));
    }
    if (static_cast<int>(threadIdx.x) < s.n_edge) {
        float lo, hi;
        f2_unpack(f(f2_pack(edge, edge)), lo, hi);
        store_scalar<ES>(s.drow + edge_column(s, threadIdx.x) * ES, lo);
    }
}

// 2^x and x with x kept above where 2^x is 0, so that 0 * x is 0; NaN passes
__device__ __forceinline__ f32x2_t clamp_exponent(f32x2_t x) {
    float lo, hi;
    f2_unpack(x, lo, hi);
    return f2_pack(max_nan(lo, kMinExp2), max_nan(hi, kMinExp2));
}

template <int ES, bool ENT>
__global__ void __launch_bounds__(kGradThreads, kGradBlocksPerSm) logprobs_grad_kernel(const RowsGradParams p) {
    griddep_launch_dependents();  // programmatic dependent launch: no global access before the wait
    griddep_wait();
    __shared__ int scratch[2 * (kGradThreads / 32)];
    if (blockIdx.x == 0 && p.err) {
        int n_valid, n_bad;
        count_labels(p.src.labels, p.src.N, p.src.V, p.src.ignore_index, scratch, n_valid, n_bad);
        if (threadIdx.x == 0) *p.err = n_bad > 0 ? FOAK_ERRBIT_LABEL_RANGE : 0;
    }
    const int64_t items = p.src.N * p.nseg;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const Segment s = segment_of<ES>(p, item);
        const int64_t y = __ldg(p.src.labels + s.row);
        if (!stream_row_valid(y, p.src)) {
            zero_segment<ES>(s);
            continue;
        }
        uint4 v[kGradVpt];
        float edge;
        load_segment<ES>(s, v, edge);
        const float2 ms = __ldg(p.stats2 + s.row);
        const float gl = (p.grad_logp ? __ldg(p.grad_logp + s.row) : 0.f) * p.inv_t;
        const float gh = ENT ? __ldg(p.grad_entropy + s.row) * p.inv_t : 0.f;
        const float hrow = ENT ? __ldg(p.entropy + s.row) : 0.f;
        const bool empty = ms.x == kNegInf;  // nothing but -inf: p = 0
        const float m = empty ? 0.f : ms.x, l2s = empty ? 0.f : ms.y * kLog2e;
        const float a = -(gl + gh * hrow), b = -gh * kLn2;
        const f32x2_t M = f2_pack(-m, -m), C = f2_pack(p.c, p.c), S = f2_pack(-l2s, -l2s);
        const f32x2_t A = f2_pack(a, a), B = f2_pack(b, b);
        const int64_t y_vec = y >= s.h && y < s.tail_col ? (y - s.h) / (16 / ES) : -1;
        float x_y = 0.f;
        const bool mine = y >= s.col_lo && y < s.col_hi &&
                          (y_vec >= 0 ? (y_vec - s.vbeg) % kGradThreads == threadIdx.x
                                      : static_cast<int>(threadIdx.x) < s.n_edge && edge_column(s, threadIdx.x) == y);
        if (mine) x_y = load_scalar<ES>(s.rowp + y * ES);
        auto grad = [&](f32x2_t x) {
            f32x2_t d = f2_fma(f2_add(x, M), C, S);  // log2 p
            if (ENT) d = clamp_exponent(d);
            return f2_mul(f2_ex2(d), ENT ? f2_fma(B, d, A) : A);
        };
        store_segment<ES>(s, v, edge, grad);
        if (mine) {  // after this thread's own store of that place
            float lo, hi;
            f2_unpack(grad(f2_pack(x_y, x_y)), lo, hi);
            store_scalar<ES>(s.drow + y * ES, lo + gl);
        }
    }
}

// Distillation: a CTA takes a run of consecutive segments, so mostly of whole rows.  A
// ninth warp fetches the teacher's row and the logits it needs before the first store of a
// row (bar `gathered`), and makes the row's corrections after the last one (`stored`),
// while the other warps are on the next row.
template <int ES, bool TWO>
__global__ void __launch_bounds__(kGradThreads + 32, kTeacherBlocksPerSm) distill_grad_kernel(const RowsGradParams p) {
    __shared__ int scratch[2 * (kGradThreads / 32 + 1)];
    __shared__ TeacherRow teacher[2];
    __shared__ uint64_t gathered[2], stored[2];
    __shared__ int s_abort;
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&gathered[i], 1);
            mbar_init(&stored[i], kGradThreads / 32);
        }
        fence_mbar_init();
        s_abort = 0;
    }
    griddep_launch_dependents();  // programmatic dependent launch: no global access before the wait
    griddep_wait();
    __syncthreads();
    int n_valid = static_cast<int>(p.src.N), n_bad = 0;
    if (p.src.labels && (!(p.denom > 0.f) || (blockIdx.x == 0 && p.err)))
        count_labels(p.src.labels, p.src.N, p.src.V, p.src.ignore_index, scratch, n_valid, n_bad);
    // The error word is 0 before the launch: each CTA adds the bits that it finds.
    if (blockIdx.x == 0 && tid == 0 && p.err && n_bad > 0)
        atomicOr(reinterpret_cast<unsigned*>(p.err), static_cast<unsigned>(FOAK_ERRBIT_LABEL_RANGE));
    const float scale = (p.g_ptr ? __ldg(p.g_ptr) : 1.f) / (p.denom > 0.f ? p.denom : static_cast<float>(n_valid));
    const float w1 = scale * p.ce_w, wt = scale * p.kd_w * p.inv_t;
    const int64_t items = p.src.N * p.nseg;
    const int64_t beg = items * blockIdx.x / gridDim.x, end = items * (blockIdx.x + 1) / gridDim.x;
    uint32_t visit = 0;  // valid rows begun
    bool aborted = false;

    // the row's plain gradient
    struct Row {
        float m, c, lt, l1, a, a1;
        __device__ __forceinline__ f32x2_t at(f32x2_t x) const {
            const f32x2_t d = f2_add(x, f2_pack(-m, -m));
            f32x2_t e = f2_mul(f2_ex2(f2_fma(d, f2_pack(c, c), f2_pack(-lt, -lt))), f2_pack(a, a));
            if (TWO) e = f2_fma(f2_ex2(f2_fma(d, f2_pack(kLog2e, kLog2e), f2_pack(-l1, -l1))), f2_pack(a1, a1), e);
            return e;
        }
    };
    auto row_of = [&](int64_t row) {
        const float4 st = __ldg(p.stats4 + row);
        const bool empty = st.x == kNegInf;  // nothing but -inf: p = 0
        Row r;
        r.m = empty ? 0.f : st.x;
        r.c = p.c;
        r.l1 = empty ? 0.f : st.y * kLog2e;
        r.lt = empty ? 0.f : st.z * kLog2e;
        r.a1 = w1;
        r.a = wt * st.w + (!TWO && p.ce_w != 0.f ? w1 : 0.f);  // one exponential where both parts share it
        return r;
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!aborted && (*reinterpret_cast<volatile int*>(&s_abort) || !mbar_wait_bounded(bar, parity, p.src.wait_ns))) {
            s_abort = 1;
            aborted = true;
        }
    };

    if (tid < kGradThreads) {
        Row r = {};
        bool valid = false;
        for (int64_t item = beg; item < end; ++item) {
            const Segment s = segment_of<ES>(p, item);
            const bool first = item == beg || s.first;
            if (first) valid = stream_row_valid(p.src.labels ? __ldg(p.src.labels + s.row) : -1, p.src);
            if (!valid) {
                zero_segment<ES>(s);
                continue;
            }
            uint4 v[kGradVpt];
            float edge;
            load_segment<ES>(s, v, edge);
            if (first) {
                r = row_of(s.row);
                wait(&gathered[visit & 1u], visit >> 1 & 1u);
                ++visit;
            }
            if (!aborted) store_segment<ES>(s, v, edge, [&](f32x2_t x) { return r.at(x); });
            if (item + 1 == end || (item + 1) % p.nseg == 0) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&stored[(visit - 1) & 1u]);
            }
        }
    } else {
        struct Visit {
            int64_t row, col_lo, col_hi, y;
            float x_y;
        } now = {}, before = {};
        bool bad_id = false;
        auto correct = [&](const Visit& u, uint32_t n) {
            wait(&stored[n & 1u], n >> 1 & 1u);
            const Row r = row_of(u.row);
            if (!aborted)
                teacher_correct<ES>(teacher[n & 1u], p.teacher.K, u.col_lo, u.col_hi, u.y, u.x_y, w1, wt,
                                    p.dx + u.row * p.src.ld * ES, [&](float x) {
                                        float lo, hi;
                                        f2_unpack(r.at(f2_pack(x, x)), lo, hi);
                                        return lo;
                                    });
            __syncwarp();
        };
        for (int64_t item = beg; item < end;) {
            Segment s = segment_of<ES>(p, item);
            const int64_t next = min(end, (s.row + 1) * p.nseg);
            now.row = s.row;
            now.y = p.src.labels ? __ldg(p.src.labels + s.row) : -1;
            if (stream_row_valid(now.y, p.src)) {
                now.col_lo = s.col_lo;
                now.col_hi = segment_of<ES>(p, next - 1).col_hi;
                bad_id |= teacher_row(p.teacher, s.row, p.src.V, teacher[visit & 1u]);
                teacher_gather<ES>(p.teacher.K, s.rowp, now.col_lo, now.col_hi, teacher[visit & 1u]);
                now.x_y = now.y >= now.col_lo && now.y < now.col_hi ? load_scalar<ES>(s.rowp + now.y * ES) : 0.f;
                __syncwarp();
                if (lane == 0) mbar_arrive(&gathered[visit & 1u]);
                if (visit > 0) correct(before, visit - 1);
                before = now;
                ++visit;
            }
            item = next;
        }
        if (visit > 0) correct(before, visit - 1);
        if (bad_id && lane == 0 && p.err)
            atomicOr(reinterpret_cast<unsigned*>(p.err), static_cast<unsigned>(FOAK_ERRBIT_LABEL_RANGE));
    }
    __syncthreads();
    if (s_abort && tid == 0 && p.err)
        atomicOr(reinterpret_cast<unsigned*>(p.err), static_cast<unsigned>(FOAK_ERRBIT_TIMEOUT));
}

RowsGradParams common_params(int es, const void* x, void* dx, int64_t ld, const int64_t* labels, int64_t N, int64_t V,
                             int64_t ignore_index, float temperature, int32_t* err) {
    RowsGradParams p = {};
    p.src.x = static_cast<const char*>(x);
    p.src.ld = ld;
    p.src.labels = labels;
    p.src.N = N;
    p.src.V = V;
    p.src.ignore_index = ignore_index;
    p.src.k = 1;
    p.src.wait_ns = test_wait_limit_ns();
    p.dx = static_cast<char*>(dx);
    p.nseg = std::max<int64_t>(1, (V * es / 16 + kGradSegVec - 1) / kGradSegVec);
    p.inv_t = 1.f / temperature;
    p.c = kLog2e / temperature;
    p.err = err;
    return p;
}

dim3 grad_grid(const RowsGradParams& p, int per_sm) {
    const int64_t full = static_cast<int64_t>(device_sm_count()) * per_sm;
    return dim3(static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(full, p.src.N * p.nseg))));
}

}  // namespace

cudaError_t launch_logprobs_grad(int es, const void* x, void* dx, int64_t ld, const int64_t* labels, int64_t N,
                                 int64_t V, int64_t ignore_index, float temperature, const float* stats,
                                 const float* grad_logp, const float* entropy, const float* grad_entropy, int32_t* err,
                                 cudaStream_t stream) {
    RowsGradParams p = common_params(es, x, dx, ld, labels, N, V, ignore_index, temperature, err);
    p.stats2 = reinterpret_cast<const float2*>(stats);
    p.entropy = entropy;
    p.grad_logp = grad_logp;
    p.grad_entropy = grad_entropy;
    const dim3 grid = grad_grid(p, kGradBlocksPerSm), block(kGradThreads);
    if (es == 2)
        return grad_entropy ? launch_dependent(logprobs_grad_kernel<2, true>, grid, block, 0, stream, p)
                            : launch_dependent(logprobs_grad_kernel<2, false>, grid, block, 0, stream, p);
    return grad_entropy ? launch_dependent(logprobs_grad_kernel<4, true>, grid, block, 0, stream, p)
                        : launch_dependent(logprobs_grad_kernel<4, false>, grid, block, 0, stream, p);
}

cudaError_t launch_distill_grad(int es, const void* x, void* dx, int64_t ld, const int64_t* labels, int64_t N,
                                int64_t V, int64_t ignore_index, const int32_t* ids, const float* logp,
                                int64_t ld_teacher, int K, bool normalize, float ce_w, float kd_w, float temperature,
                                const float* stats, const float* grad_out, float denom, int32_t* err,
                                cudaStream_t stream) {
    RowsGradParams p = common_params(es, x, dx, ld, labels, N, V, ignore_index, temperature, err);
    p.stats4 = reinterpret_cast<const float4*>(stats);
    p.teacher.ids = ids;
    p.teacher.logp = logp;
    p.teacher.ld = ld_teacher;
    p.teacher.K = K;
    p.teacher.normalize = normalize;
    p.g_ptr = grad_out;
    p.denom = denom;
    p.ce_w = ce_w;
    p.kd_w = kd_w;
    // Any CTA may have a bit for the error word, and no memory here is known to be 0 for a count
    // of those that are done: so the word is cleared by a step of its own (515 x 49159 fp32, the
    // backward alone: 42.8 -> 45.8 us; behind its forward, which it no longer starts under, 69.8 -> 65.3).
    if (err) {
        const cudaError_t e = cudaMemsetAsync(err, 0, sizeof(int32_t), stream);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid = grad_grid(p, kTeacherBlocksPerSm), block(kGradThreads + 32);
    const bool two = ce_w != 0.f && temperature != 1.f;
    if (es == 2)
        return two ? launch_dependent(distill_grad_kernel<2, true>, grid, block, 0, stream, p)
                   : launch_dependent(distill_grad_kernel<2, false>, grid, block, 0, stream, p);
    return two ? launch_dependent(distill_grad_kernel<4, true>, grid, block, 0, stream, p)
               : launch_dependent(distill_grad_kernel<4, false>, grid, block, 0, stream, p);
}

}  // namespace foak
