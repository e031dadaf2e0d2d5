// Distillation from a teacher's top tokens over rows of student logits: the loss, and
// (fused) its gradient.  With T the temperature, p = softmax(x / T), q the teacher's
// probabilities of its K listed tokens (renormalised, or as they are) and y the label:
//
//   KD = sum_k q_k (ln q_k - ln p_{id_k})      CE = ln sum_j e^{x_j} - x_y
//   loss = sum over valid rows (w_ce CE + w_kd KD) / D
//   dx_j = (g / D) (w_ce (softmax(x)_j - [j = y]) + (w_kd / T) (Q p_j - sum_k q_k [j = id_k])),  Q = sum_k q_k
//
// The gradient is the softmax of the whole row times a constant, except at K + 1 places.
// So the kernel is a row kernel with two sweeps -- sums, then gradient -- whose second
// one writes a1 e^{x - m} + aT e^{(x - m) / T} everywhere, after which a closing warp
// overwrites the K + 1 places (from logits fetched before the sweep began, so that the
// gradient may replace the logits) while the others are on the next row.  The second sweep
// re-reads the row from L2: HBM sees each logit read once and written once.  T = 1, or no
// cross-entropy part, needs one exponential an element; otherwise there are two sums and
// two exponentials.
//
// Measured, bf16: 8192 x 128256, K = 128, loss and gradient 667 us (6.15 TB/s read and
// written); 4096 x 32000, K = 64: 96 us at T = 1 (5.5 TB/s), 117 at T = 2 with a cross-entropy
// part; the loss alone 53 and 62.  HBM bounds the long rows; the short ones at
// T = 2 take two exponentials an element and sweep (64% of the issue slots) and wait between a
// row's two sweeps.
#include <algorithm>

#include "row_stream.cuh"
#include "teacher.cuh"

namespace foak {

namespace {

struct DistillParams {
    StreamSrc src;
    CeRowParams fin;   // what the shared end of the row kernels takes: loss terms, denominator, workspace
    TeacherSrc teacher;
    char* dx;
    float ce_w, kd_w;
    float inv_t;       // 1 / T
    ExpScale scale;
    float g;
    float* row_ce;     // [N] or null
    float* row_kd;     // [N] or null
    float4* stats;     // [N] or null: (m, ln sum e^(x-m), ln sum e^((x-m)/T), Q)
};

// What the second sweep works with: the maximum, and the factors of the two exponentials.
struct SweepFactors {
    float m, a, a1;
};
template <bool TWO>
__device__ __forceinline__ SweepFactors sweep_factors(const RunStat<false, TWO>& st, float total, float w1, float wt) {
    const float s1 = TWO ? st.s2 : st.s;  // at T = 1 they are the same; without w_ce it is not used
    SweepFactors f;
    f.m = st.m;
    const float at = st.s == 0.f ? 0.f : wt * total / st.s;  // nothing but -inf: p = 0
    f.a1 = w1 != 0.f && s1 != 0.f ? w1 / s1 : 0.f;
    f.a = TWO ? at : at + f.a1;
    return f;
}

// Closing warps of a CTA, which take rows in turn: one is still at a row's corrections when the
// next row's targets are wanted.
constexpr int kClosers = 2;
template <int NT>
constexpr int kDistillThreads = NT + 32 + 32 * kClosers;

template <int ES, bool GRAD, bool TWO, int NT>
__global__ void __launch_bounds__(kDistillThreads<NT>, NT == 256 ? 2 : 1) distill_kernel(const DistillParams p) {
    constexpr int EPV = 16 / ES;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ StreamBars bars;
    __shared__ StatExchange ex;
    __shared__ LongSums aside;
    __shared__ TeacherRow teacher[kClosers];
    __shared__ SweepFactors factors[kMaxBuffers];
    __shared__ float total[kMaxBuffers];  // of the teacher's row
    __shared__ int s_count[kMaxWarps];
    __shared__ int s_valid;  // valid rows of the call, for the scale: written once, read by the closing warps at any time
    __shared__ int s_rows, s_bad, s_last;  // valid rows of this CTA
    __shared__ DFloat dred[kDistillThreads<NT> / 32];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = p.src.k;
    const int rank = k > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int64_t cid = blockIdx.x >> p.src.log2_k, ncl = gridDim.x >> p.src.log2_k;
    const int64_t n_it = stream_rows(p.src, cid);
    stream_init<NT>(bars, p.src.stages, k);
    if (tid == 0) s_bad = 0;
    griddep_launch_dependents();  // programmatic dependent launch: no global access before the wait
    griddep_wait();
    // the producer's and closing warps' first 32 rows, the consumers' first one
    const int64_t label0 = first_label(p.src, cid, ncl, warp < Shape<NT>::kWarps ? 0 : lane);
    __syncthreads();
    if (k > 1) cluster_arrive_release();  // waited for before the cluster's memory is written to

    const ExpScale& sc = p.scale;
    if (warp == Shape<NT>::kWarps) {
        stream_produce<ES, NT>(p.src, bars, smem, GRAD ? 2 : 1, cid, ncl, rank, label0);
        if (k > 1) cluster_wait_acquire();
    } else if (warp < Shape<NT>::kWarps) {
        float scale = 0.f;
        if (GRAD) {
            scale = p.g / p.fin.denom;
            if (!(p.fin.denom > 0.f)) {
                const int n = count_valid_consumers<NT>(p.src, s_count);
                scale = p.g / static_cast<float>(n);
                if (tid == 0) s_valid = n;
                scale_known<NT, kClosers>();
            }
        }
        StreamPos pos{0, 0, false};
        RowPos rp;
        Slice s = slice_of<ES>(p.src, cid, rank);
        int64_t y_next = label0;
        for (int64_t it = 0; it < n_it; ++it) {
            const int64_t row = cid + it * ncl;
            const int64_t y = y_next;
            if (p.src.labels && it + 1 < n_it) y_next = __ldg(p.src.labels + row + ncl);
            move_slice<ES>(p.src, row, rank, s);
            char* drow = p.dx + row * p.src.ld * ES;
            uint4* dv = reinterpret_cast<uint4*>(drow + s.col0 * ES);
            if (!stream_row_valid(y, p.src)) {
                if constexpr (GRAD) {
                    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
                    for (int i = tid; i < s.nv; i += NT) st_global_cs_v4(dv + i, z);
                    if (tid < s.h) store_scalar<ES>(drow + tid * ES, 0.f);
                    if (tid < s.t) store_scalar<ES>(drow + (s.tail_col + tid) * ES, 0.f);
                }
                continue;
            }
            row_begin(p.src, bars, rp, pos);
            RunStat<false, TWO> st(sc);
            for (int run = 0; run < s.nv; run += kRunVec<NT>) {
                if (run > 0) {
                    stat_put_aside<false, TWO>(st, aside, run == kRunVec<NT>, sc);
                    st.restart();
                }
                const int end = min(s.nv, run + kRunVec<NT>);
                for (int c0 = run; c0 < end; c0 += Shape<NT>::kChunk) {
                    const int nl = min(Shape<NT>::kChunk, s.nv - c0);
                    uint4 v[kBlockVec];
                    stream_chunk<NT>(p.src, bars, smem, pos, [&](const unsigned char* stage) { load_strided<ES, NT>(stage, nl, v); });
                    st.template add_vecs<ES>(v, sc);
                }
            }
            // the head and tail scalars, one a lane of the first warp; kept for the gradient
            const int n_edge = s.h + s.t;
            const int64_t edge_col = tid < s.h ? tid : s.tail_col + (tid - s.h);
            float edge = kNegInf;
            if (n_edge > 0 && warp == 0) {
                if (tid < n_edge) edge = load_scalar<ES>(s.rowp + edge_col * ES);
                st.add(edge, sc);
            }
            const int buf = rp.buf;
            if (s.nv <= kRunVec<NT>) stat_publish(st, ex, buf);
            else stat_publish_long(st, aside, ex, buf, sc);
            row_end(bars, buf);
            if constexpr (GRAD) {
                if (!pos.aborted && !stream_wait(bars, &bars.row_ready[buf], rp.use & 1u, p.src.wait_ns))
                    pos.aborted = true;
                SweepFactors f;
                if (k == 1) {
                    // Every warp joins the row's sums for itself: no way to the closing warp and back.
                    if (!pos.aborted && !stream_wait(bars, &bars.row_full[buf], rp.use & 1u, p.src.wait_ns))
                        pos.aborted = true;
                    stat_collect<NT>(st, ex, buf, sc);
                    st.correct(sc);
                    f = sweep_factors(st, total[buf], scale * p.ce_w, scale * p.kd_w * p.inv_t);
                } else {
                    f = factors[buf];
                }
                const f32x2_t M = f2_pack(-f.m, -f.m), C = f2_pack(sc.c, sc.c), L = f2_pack(kLog2e, kLog2e);
                const f32x2_t A = f2_pack(f.a, f.a), A1 = f2_pack(f.a1, f.a1);
                auto grad = [&](f32x2_t x) {
                    const f32x2_t d = f2_add(x, M);
                    f32x2_t e = f2_mul(f2_ex2(f2_mul(d, C)), A);
                    if (TWO) e = f2_fma(f2_ex2(f2_mul(d, L)), A1, e);
                    return e;
                };
                for (int c0 = 0; c0 < s.nv; c0 += Shape<NT>::kChunk) {
                    const int nl = min(Shape<NT>::kChunk, s.nv - c0);
                    uint4 v[kBlockVec];
                    stream_chunk<NT>(p.src, bars, smem, pos, [&](const unsigned char* stage) { load_strided<ES, NT>(stage, nl, v); });
                    if (pos.aborted) continue;
#pragma unroll
                    for (int i = 0; i < kBlockVec; ++i) {
                        uint32_t o[4];
#pragma unroll
                        for (int j = 0; j < EPV / 2; ++j) {
                            const f32x2_t e = grad(vec_pair<ES>(v[i], j));
                            if constexpr (ES == 2) {
                                o[j] = f2_to_bf16x2(e);
                            } else {
                                float lo, hi;
                                f2_unpack(e, lo, hi);
                                o[2 * j] = __float_as_uint(lo);
                                o[2 * j + 1] = __float_as_uint(hi);
                            }
                        }
                        const int lv = tid + i * NT;
                        if (nl == Shape<NT>::kChunk || lv < nl) st_global_cs_v4(dv + c0 + lv, make_uint4(o[0], o[1], o[2], o[3]));
                    }
                }
                if (tid < n_edge && !pos.aborted) {
                    float lo, hi;
                    f2_unpack(grad(f2_pack(edge, edge)), lo, hi);
                    store_scalar<ES>(drow + edge_col * ES, lo);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.row_stored[buf]);
            }
            rp.next(p.src);
        }
        __syncwarp();
        if (k > 1) cluster_wait_acquire();
    } else {  // a closing warp
        if (k > 1) cluster_wait_acquire();
        const int me = warp - (Shape<NT>::kWarps + 1);  // buffer `me` is this warp's
        TeacherRow& teach = teacher[me];
        float scale = 0.f;
        if (GRAD) {
            if (!(p.fin.denom > 0.f)) scale_known<NT, kClosers>();
            scale = p.g / (p.fin.denom > 0.f ? p.fin.denom : static_cast<float>(s_valid));
        }
        const float w1 = scale * p.ce_w, wt = scale * p.kd_w * p.inv_t;
        const int K = p.teacher.K;
        RowPos rp;
        Slice s = slice_of<ES>(p.src, cid, rank);
        int n_bad = 0;
        bool aborted = false;
        for (int64_t base = 0; base < n_it; base += 32) {
            // 32 rows' labels at once, and the logits of this warp's rows, a row a lane.  (A row's gradient is
            // not begun before its closing warp has made it ready, so the logits are still there.)
            int64_t lab = label0;
            bool ok = false;
            if (base + lane < n_it) {
                if (base > 0 && p.src.labels) lab = __ldg(p.src.labels + cid + (base + lane) * ncl);
                ok = stream_row_valid(lab, p.src);
                n_bad += !ok && lab != p.src.ignore_index && me == 0;
            }
            const unsigned valid = __ballot_sync(0xffffffffu, ok);
            float x_lab = 0.f;
            if (p.src.labels && ok && (rp.buf + __popc(valid & ((1u << lane) - 1u))) % kClosers == me)
                x_lab = load_scalar<ES>(p.src.x + ((cid + (base + lane) * ncl) * p.src.ld + lab) * ES);
            const int nj = static_cast<int>(min(static_cast<int64_t>(32), n_it - base));
            for (int j = 0; j < nj; ++j) {
                const int64_t row = cid + (base + j) * ncl;
                if (!(valid >> j & 1u)) {
                    if (rank == 0 && me == 0 && lane == 0) {
                        p.fin.row_loss[row] = 0.f;
                        if (p.row_ce) p.row_ce[row] = 0.f;
                        if (p.row_kd) p.row_kd[row] = 0.f;
                        if (p.stats) p.stats[row] = make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                    continue;
                }
                if (rp.buf != me) {
                    rp.next(p.src);
                    continue;
                }
                const int64_t y = p.src.labels ? __shfl_sync(0xffffffffu, lab, j) : -1;
                const float x_y = __shfl_sync(0xffffffffu, x_lab, j);
                const int buf = rp.buf;
                const uint32_t use = rp.use;
                move_slice<ES>(p.src, row, rank, s);
                const int64_t col_lo = rank == 0 ? 0 : s.col0;
                const int64_t col_hi = rank == k - 1 ? p.src.V : s.col0 + static_cast<int64_t>(s.nv) * EPV;
                const bool bad = teacher_row(p.teacher, row, p.src.V, teach);
                n_bad += bad && lane == 0;
                // Rank 0 takes all the listed logits (for the loss), the others those of their share: ahead of
                // the row where its gradient may overwrite it, else after it, when they are in L2 (4096 x 32000
                // bf16, K = 64: 52.6 us, ahead of it 57.7; with the gradient both took 96).
                auto gather = [&] {
                    teacher_gather<ES>(K, s.rowp, rank == 0 ? 0 : col_lo, rank == 0 ? p.src.V : col_hi, teach);
                };
                if (GRAD) gather();
                if (GRAD && k == 1 && lane == 0) {  // all that the second sweep needs from here
                    total[buf] = teach.total;
                    mbar_arrive(&bars.row_ready[buf]);
                }
                if (!aborted && !stream_wait(bars, &bars.row_full[buf], use & 1u, p.src.wait_ns)) aborted = true;
                if (!GRAD) gather();
                RunStat<false, TWO> st(sc);
                stat_collect<NT>(st, ex, buf, sc);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.row_empty[buf]);
                if (k > 1) {
                    stat_send(st, ex, k, rank);
                    if (!peers_meet(bars, k, aborted ? 0 : p.src.wait_ns)) aborted = true;
                    stat_merge(st, ex, k, sc);
                }
                st.correct(sc);
                const bool empty = st.s == 0.f;  // nothing but -inf: every token's log probability is -inf
                const float s1 = TWO ? st.s2 : st.s;
                const SweepFactors f = sweep_factors(st, teach.total, w1, wt);
                if (GRAD && k > 1 && lane == 0) {
                    factors[buf] = f;
                    mbar_arrive(&bars.row_ready[buf]);
                }
                if (rank == 0 && !aborted) {
                    const float ln_t = logf(st.s), ln_1 = logf(s1);
                    float kd = 0.f;
#pragma unroll 1
                    for (int i = lane; i < K; i += 32) {
                        const float q = teach.q[i];
                        if (!(q == 0.f)) kd += q * (teach.lnq[i] - (empty ? kNegInf : (teach.x[i] - st.m) * p.inv_t - ln_t));
                    }
                    kd = warp_sum(kd);
                    if (lane == 0) {
                        const float ce = p.ce_w != 0.f ? (empty ? -kNegInf : ln_1 - (x_y - st.m)) : 0.f;
                        p.fin.row_loss[row] = (p.ce_w != 0.f ? p.ce_w * ce : 0.f) + (p.kd_w != 0.f ? p.kd_w * kd : 0.f);
                        if (p.row_ce) p.row_ce[row] = ce;
                        if (p.row_kd) p.row_kd[row] = kd;
                        if (p.stats) p.stats[row] = make_float4(empty ? kNegInf : st.m, ln_1, ln_t, teach.total);
                    }
                }
                if constexpr (GRAD) {
                    // The K + 1 places that differ, after the consumers' stores of the row.
                    if (!aborted && !stream_wait(bars, &bars.row_stored[buf], use & 1u, p.src.wait_ns)) aborted = true;
                    if (!aborted) {
                        teacher_correct<ES>(teach, K, col_lo, col_hi, y, x_y, w1, wt, p.dx + row * p.src.ld * ES, [&](float x) {
                            const float d = x - f.m;
                            float e = ex2(d * sc.c) * f.a;
                            if (TWO) e = fmaf(ex2(d * kLog2e), f.a1, e);
                            return e;
                        });
                    }
                }
                __syncwarp();
                rp.next(p.src);
            }
        }
        n_bad = __reduce_add_sync(0xffffffffu, n_bad);
        if (lane == 0) {
            if (me == 0) s_rows = rank == 0 ? static_cast<int>(rp.n) : 0;
            if (rank == 0 && n_bad) atomicAdd(&s_bad, n_bad);
            if (aborted) bars.abort = 1;
        }
    }
    __syncthreads();
    rows_finish<kDistillThreads<NT>>(p.fin, stream_aborted(bars), s_rows, s_bad, &s_last, dred, true);
    if (k > 1) cluster_sync_converged();  // no CTA leaves while its shared memory may be written
}

template <int ES, bool GRAD, bool TWO, int NT>
cudaError_t launch_typed(DistillParams prm, int per_sm, cudaStream_t stream) {
    auto* kern = &distill_kernel<ES, GRAD, TWO, NT>;
    StreamSrc& s = prm.src;
    s.buffers = kClosers;
    const size_t fixed = 1024 + 512 + sizeof(StreamBars) + sizeof(StatExchange) + sizeof(LongSums) +
                         kClosers * sizeof(TeacherRow);
    const size_t room = std::min<size_t>((228 * 1024) / per_sm, 227 * 1024) - fixed;
    s.stages = static_cast<int>(std::min<size_t>(kStreamMaxStages, room / Shape<NT>::kStageBytes));
    const size_t smem = static_cast<size_t>(s.stages) * Shape<NT>::kStageBytes;
    static SmemLimit limit;
    const cudaError_t e = limit.allow(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    const int64_t clusters = std::max<int64_t>(1, std::min<int64_t>(s.N, static_cast<int64_t>(device_sm_count()) * per_sm / s.k));
    if (!set_rows(s, clusters)) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * s.k), 1, 1);
    cfg.blockDim = dim3(kDistillThreads<NT>, 1, 1);
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

template <int ES, bool GRAD, bool TWO>
cudaError_t launch_shape(DistillParams p, cudaStream_t stream) {
    StreamSrc& s = p.src;
    const int sms = device_sm_count();
    // One CTA an SM: 130 fused rows of 128256 bf16 by 1, 2, 4 and 8 took 21.6, 23.8, 27.6 and
    // 42.9 us, 16 rows 18.8, 16.4, 12.2 and 12.2.
    const int k = cluster_size(s, ES, 8 * 1024, sms);
    set_cluster(s, k);
    int per_sm = 2;
    if constexpr (GRAD) {
        // The rows between their two sweeps wait in L2 (129 MB, which the gradient's lines share): two CTAs
        // an SM while those rows stay within 64 MB (4096 x 32000 bf16, T = 2: 125 us, one CTA of 512 threads
        // 149), then one CTA of twice the threads (8192 x 128256: 663 us, of 256 threads with two CTAs of a
        // cluster 785).
        while (per_sm > 1 && static_cast<double>(sms) * per_sm / k * static_cast<double>(s.V) * ES > 64e6) --per_sm;
        s.evict_last_pass = true;
        if (per_sm == 1 && k == 1) return launch_typed<ES, GRAD, TWO, 512>(p, 1, stream);
    }
    return launch_typed<ES, GRAD, TWO, 256>(p, per_sm, stream);
}

template <int ES, bool GRAD>
cudaError_t launch_two(const DistillParams& p, float temperature, cudaStream_t stream) {
    // a second sum only where both parts are wanted at different temperatures
    return p.ce_w != 0.f && temperature != 1.f ? launch_shape<ES, GRAD, true>(p, stream)
                                               : launch_shape<ES, GRAD, false>(p, stream);
}

}  // namespace

cudaError_t launch_distill(bool grad, int es, const void* x, void* dx, int64_t ld, const int64_t* labels, int64_t N,
                           int64_t V, int64_t ignore_index, const int32_t* ids, const float* logp, int64_t ld_teacher,
                           int K, bool normalize, float ce_w, float kd_w, float temperature, float g, float denom,
                           float* loss, float* row_loss, float* row_ce, float* row_kd, float* stats, int32_t* n_valid,
                           int32_t* err, CeWsHeader* ws, cudaStream_t stream) {
    DistillParams p = {};
    p.src.x = static_cast<const char*>(x);
    p.src.ld = ld;
    p.src.labels = labels;
    p.src.N = N;
    p.src.V = V;
    p.src.ignore_index = ignore_index;
    p.src.wait_ns = test_wait_limit_ns();
    p.src.skip_load_row = test_skip_load_row();
    p.fin.N = N;
    p.fin.denom = denom;
    p.fin.loss = loss;
    p.fin.row_loss = row_loss;
    p.fin.n_valid = n_valid;
    p.fin.err = err;
    p.fin.ws = ws;
    p.teacher.ids = ids;
    p.teacher.logp = logp;
    p.teacher.ld = ld_teacher;
    p.teacher.K = K;
    p.teacher.normalize = normalize;
    p.dx = static_cast<char*>(dx);
    p.ce_w = ce_w;
    p.kd_w = kd_w;
    p.inv_t = 1.f / temperature;
    p.scale = exp_scale(temperature);
    p.g = g;
    p.row_ce = row_ce;
    p.row_kd = row_kd;
    p.stats = reinterpret_cast<float4*>(stats);
    if (es == 2) return grad ? launch_two<2, true>(p, temperature, stream) : launch_two<2, false>(p, temperature, stream);
    return grad ? launch_two<4, true>(p, temperature, stream) : launch_two<4, false>(p, temperature, stream);
}

}  // namespace foak
