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
// one writes a1 e^{x - m} + aT e^{(x - m) / T} everywhere, after which the K + 1 places
// are overwritten (after a barrier, from logits kept when the row began, so that the
// gradient may replace the logits).  The second sweep re-reads the row from L2: HBM sees
// each logit read once and written once.  T = 1, or no cross-entropy part, needs one
// exponential an element; otherwise there are two sums and two exponentials.
#include <algorithm>
#include <map>
#include <mutex>

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

template <int ES, bool GRAD, bool TWO>
__global__ void __launch_bounds__(kStreamBlock, 3) distill_kernel(const DistillParams p) {
    constexpr int EPV = 16 / ES;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ StreamBars bars;
    __shared__ StatExchange ex;
    __shared__ TeacherRow teach;
    __shared__ float s_xy;
    __shared__ int s_count[kStreamWarps];
    __shared__ int s_last;
    __shared__ DFloat dred[kStreamBlock / 32];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = p.src.k;
    const int rank = k > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int64_t cid = blockIdx.x / k, ncl = gridDim.x / k;
    const int64_t n_it = p.src.N > cid ? (p.src.N - 1 - cid) / ncl + 1 : 0;
    stream_init(bars, p.src.stages);
    griddep_launch_dependents();  // programmatic dependent launch: no global access before the wait
    griddep_wait();
    __syncthreads();
    if (k > 1) cluster_sync();

    int n_valid = 0, n_bad = 0;
    bool aborted = false;
    if (tid >= kStreamThreads) {
        stream_produce<ES>(p.src, bars, smem, GRAD ? 2 : 1, cid, ncl, rank, k > 1 ? 1 : 0);
    } else {
        float scale = 0.f;
        if constexpr (GRAD) {
            const bool given = p.fin.denom > 0.f;
            scale = p.g / (given ? p.fin.denom : static_cast<float>(count_valid_consumers(p.src, s_count)));
        }
        const float w1 = scale * p.ce_w, wt = scale * p.kd_w * p.inv_t;
        StreamPos pos{0, 0, false};
        Slice s = slice_of<ES>(p.src, cid, rank);
        uint32_t parity = 0;
        int64_t y_next = p.src.labels && n_it > 0 ? __ldg(p.src.labels + cid) : 0;
        for (int64_t it = 0; it < n_it; ++it) {
            const int64_t row = cid + it * ncl;
            const int64_t y = y_next;
            if (p.src.labels && it + 1 < n_it) y_next = __ldg(p.src.labels + row + ncl);
            move_slice<ES>(p.src, row, rank, s);
            char* drow = GRAD ? p.dx + row * p.src.ld * ES : nullptr;
            uint4* dv = reinterpret_cast<uint4*>(drow + s.col0 * ES);
            if (!stream_row_valid(y, p.src)) {
                if (rank == 0 && tid == 0) {
                    n_bad += y != p.src.ignore_index;
                    p.fin.row_loss[row] = 0.f;
                    if (p.row_ce) p.row_ce[row] = 0.f;
                    if (p.row_kd) p.row_kd[row] = 0.f;
                    if (p.stats) p.stats[row] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
                if constexpr (GRAD) {
                    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
                    for (int i = tid; i < s.nv; i += kStreamThreads) st_global_cs_v4(dv + i, z);
                    if (tid < s.h) store_scalar<ES>(drow + tid * ES, 0.f);
                    if (tid < s.t) store_scalar<ES>(drow + (s.tail_col + tid) * ES, 0.f);
                }
                continue;
            }
            const int64_t col_lo = rank == 0 ? 0 : s.col0;
            const int64_t col_hi = rank == k - 1 ? p.src.V : s.col0 + static_cast<int64_t>(s.nv) * EPV;
            if (warp == 0) {
                // rank 0 takes all the listed logits (for the loss), the others those of their share
                const bool bad = teacher_row<ES>(p.teacher, row, p.src.V, s.rowp, rank == 0 ? 0 : col_lo,
                                                 rank == 0 ? p.src.V : col_hi, teach);
                if (lane == 0) {
                    s_xy = p.src.labels ? load_scalar<ES>(s.rowp + y * ES) : 0.f;
                    if (rank == 0) {
                        ++n_valid;
                        n_bad += bad;
                    }
                }
            }
            RunStat<false, TWO> st(p.scale);
            for (int c0 = 0; c0 < s.nv; c0 += kStreamChunk) {
                const int nl = min(kStreamChunk, s.nv - c0);
                uint4 v[kBlockVec];
                stream_chunk(p.src, bars, smem, pos, [&](const unsigned char* stage) { load_strided<ES>(stage, nl, v); });
                st.template add_vecs<ES>(v, p.scale);
            }
            // the head and tail scalars, one a thread; kept for the gradient
            const int n_edge = s.h + s.t;
            const int64_t edge_col = tid < s.h ? tid : s.tail_col + (tid - s.h);
            float edge = kNegInf;
            if (n_edge > 0 && tid < 32) {
                if (tid < n_edge) edge = load_scalar<ES>(s.rowp + edge_col * ES);
                st.add(edge, p.scale);
            }
            stat_publish(st, ex, parity);
            consumers_sync();
            stat_collect(st, ex, parity, p.scale);
            if (k > 1) {
                stat_send(st, ex, parity, k, rank);
                cluster_sync_converged();
                stat_merge(st, ex, parity, k, p.scale);
            }
            st.correct(p.scale);
            parity ^= 1u;
            const float s1 = TWO ? st.s2 : st.s;  // at T = 1 they are the same; without w_ce it is not used
            if (rank == 0 && warp == 0 && !pos.aborted) {
                const bool empty = st.s == 0.f;  // nothing but -inf: every token has log probability -inf
                const float ln_t = logf(st.s), ln_1 = logf(s1);
                float kd = 0.f;
                for (int j = lane; j < p.teacher.K; j += 32) {
                    const float q = teach.q[j];
                    if (!(q == 0.f)) kd += q * (teach.lnq[j] - (empty ? kNegInf : (teach.x[j] - st.m) * p.inv_t - ln_t));
                }
                kd = warp_sum(kd);
                if (lane == 0) {
                    const float ce = p.ce_w != 0.f ? (empty ? -kNegInf : ln_1 - (s_xy - st.m)) : 0.f;
                    p.fin.row_loss[row] = (p.ce_w != 0.f ? p.ce_w * ce : 0.f) + (p.kd_w != 0.f ? p.kd_w * kd : 0.f);
                    if (p.row_ce) p.row_ce[row] = ce;
                    if (p.row_kd) p.row_kd[row] = kd;
                    if (p.stats) p.stats[row] = make_float4(st.s == 0.f ? kNegInf : st.m, ln_1, ln_t, teach.total);
                }
            }
            if constexpr (GRAD) {
                // a row of -inf alone has p = 0
                const float at = st.s == 0.f ? 0.f : wt * teach.total / st.s;
                const float a1 = p.ce_w != 0.f && s1 != 0.f ? w1 / s1 : 0.f;
                const float a = TWO ? at : at + a1;
                const f32x2_t M = f2_pack(-st.m, -st.m), C = f2_pack(p.scale.c, p.scale.c), L = f2_pack(kLog2e, kLog2e);
                const f32x2_t A = f2_pack(a, a), A1 = f2_pack(a1, a1);
                for (int c0 = 0; c0 < s.nv; c0 += kStreamChunk) {
                    const int nl = min(kStreamChunk, s.nv - c0);
                    uint4 v[kBlockVec];
                    stream_chunk(p.src, bars, smem, pos, [&](const unsigned char* stage) { load_strided<ES>(stage, nl, v); });
                    if (pos.aborted) continue;
#pragma unroll
                    for (int i = 0; i < kBlockVec; ++i) {
                        uint32_t o[4];
#pragma unroll
                        for (int j = 0; j < EPV / 2; ++j) {
                            const f32x2_t d = f2_add(vec_pair<ES>(v[i], j), M);
                            f32x2_t e = f2_mul(f2_ex2(f2_mul(d, C)), A);
                            if (TWO) e = f2_fma(f2_ex2(f2_mul(d, L)), A1, e);
                            if constexpr (ES == 2) {
                                o[j] = f2_to_bf16x2(e);
                            } else {
                                float lo, hi;
                                f2_unpack(e, lo, hi);
                                o[2 * j] = __float_as_uint(lo);
                                o[2 * j + 1] = __float_as_uint(hi);
                            }
                        }
                        const int lv = tid + i * kStreamThreads;
                        if (lv < nl) st_global_cs_v4(dv + c0 + lv, make_uint4(o[0], o[1], o[2], o[3]));
                    }
                }
                auto grad_at = [&](float x) {
                    const float d = x - st.m;
                    float e = ex2(d * p.scale.c) * a;
                    if (TWO) e = fmaf(ex2(d * kLog2e), a1, e);
                    return e;
                };
                if (tid < n_edge && !pos.aborted) store_scalar<ES>(drow + edge_col * ES, grad_at(edge));
                consumers_sync();  // every plain store of this CTA is made: the places that differ may follow
                for (int j = tid; j <= p.teacher.K; j += kStreamThreads) {
                    const bool is_label = j == p.teacher.K;
                    if (is_label && !p.src.labels) continue;
                    const int64_t id = is_label ? y : teach.id[j];
                    if (id < 0 || id < col_lo || id >= col_hi || pos.aborted) continue;
                    // a token listed twice, or listed and the label, gets the same value from each
                    float e = grad_at(is_label ? s_xy : teach.x[j]) - wt * teacher_mass(teach, p.teacher.K, static_cast<int>(id));
                    if (p.src.labels && id == y) e -= w1;
                    store_scalar<ES>(drow + id * ES, e);
                }
            }
            consumers_sync();  // the teacher's row may be overwritten
        }
        aborted = pos.aborted;
    }
    __syncthreads();
    rows_finish<kStreamBlock>(p.fin, aborted || stream_aborted(bars), n_valid, n_bad, &s_last, dred, true);
    if (k > 1) cluster_sync_converged();  // no CTA leaves while its shared memory may be written
}

std::mutex g_ds_mu;
std::map<std::pair<int, const void*>, size_t> g_ds_attr;  // (device, kernel): dynamic shared memory allowed

template <int ES, bool GRAD, bool TWO>
cudaError_t launch_typed(DistillParams prm, cudaStream_t stream) {
    auto* kern = &distill_kernel<ES, GRAD, TWO>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    StreamSrc& s = prm.src;
    const int sms = device_sm_count();
    const int64_t nb = s.V * ES / 16 + 1;
    int k = kStreamMaxCluster;
    while (k > 1 && (s.N * k > sms || 2 * nb < static_cast<int64_t>(k) * kStreamChunk)) k /= 2;
    set_cluster(s, k);
    const size_t fixed = 1024 + sizeof(StreamBars) + sizeof(StatExchange) + sizeof(TeacherRow) + 512;
    const int per_sm = 3;
    const size_t room = (228 * 1024) / per_sm - fixed;
    s.stages = static_cast<int>(std::min<size_t>(kStreamMaxStages, room / kStreamStageBytes));
    const size_t smem = static_cast<size_t>(s.stages) * kStreamStageBytes;
    {
        std::lock_guard<std::mutex> lock(g_ds_mu);
        size_t& set = g_ds_attr[std::make_pair(dev, reinterpret_cast<const void*>(kern))];
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

template <int ES, bool GRAD>
cudaError_t launch_two(const DistillParams& p, float temperature, cudaStream_t stream) {
    // a second sum only where both parts are wanted at different temperatures
    return p.ce_w != 0.f && temperature != 1.f ? launch_typed<ES, GRAD, true>(p, stream)
                                               : launch_typed<ES, GRAD, false>(p, stream);
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
