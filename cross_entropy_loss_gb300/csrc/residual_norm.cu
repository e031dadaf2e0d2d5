// A block's output joins the residual stream, and the next block's input is normalised:
//     u = X  or  X r1 gp,  r1 = 1 / sqrt(mean X^2 + eps_p)          (the norm after a block)
//     h = R + s g u,       r = 1 / sqrt(mean h^2 + eps),   y = h r gamma
// with a residual scale s and a gate g that is absent, one a channel, one a row or one an
// element.  The arithmetic is fp32; h and y are rounded once each, y from the unrounded h.
//
// Backward, from the rounded h, r and r1 (hh = h r, t = gamma dy, xh = X r1, e the gate):
//     dh = dH + r (t - hh mean(hh t)),   dR = dh,   dgamma = sum_i dy hh
//     du = s e dh,   dg = s dh u summed over what shares g
//     dX = du  or  r1 (gp du - xh mean(xh gp du)),   dgp = sum_i du xh
//
// Both directions are bound by memory: each operand is read and each result written once.
#include <algorithm>
#include <mutex>

#include "foak_ce.h"
#include "internal.h"
#include "residual_norm.h"
#include "vec16.cuh"

namespace foak {

namespace {

// Sum over the CTA in a fixed order (a tree a warp, then the same tree over the warps); every
// thread gets it.  `red` has 32 floats; two calls in a row need different ones.
__device__ __forceinline__ float block_sum(float v, float* red) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return warp_sum(lane < static_cast<int>(blockDim.x >> 5) ? red[lane] : 0.f);
}

// Rows of any length up to kResNormMaxD, a CTA a row: h stays in shared memory as floats between
// the sum of its squares and y.
template <int ES>
__global__ void __launch_bounds__(512) resnorm_fwd_row_kernel(const ResNormFwd a) {
    griddep_launch_dependents();  // programmatic dependent launch: no global access before the wait
    griddep_wait();
    using V = Vec16<ES>;
    extern __shared__ float row_h[];
    __shared__ float red[2][32];
    const int nvec = static_cast<int>(a.D / V::N);
    const float inv_d = 1.f / static_cast<float>(a.D);
    for (int64_t i = blockIdx.x; i < a.N; i += gridDim.x) {
        const char* x = a.X + i * a.ldx * ES;
        const char* r = a.R + i * a.ldr * ES;
        const char* g = a.gate_kind == FOAK_GATE_CHANNEL ? a.gate : a.gate + i * a.ldg * ES;
        float q = a.scale;
        if (a.gate_kind == FOAK_GATE_ROW) q *= V::load1(g);
        if (a.post_gamma) {
            float ss = 0.f;
            for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
                float f[V::N];
                V::load(x + v * 16, f);
#pragma unroll
                for (int k = 0; k < V::N; ++k) ss = fmaf(f[k], f[k], ss);
            }
            const float r1 = rsqrtf(block_sum(ss, red[0]) * inv_d + a.post_eps);
            if (threadIdx.x == 0 && a.post_rstd) a.post_rstd[i] = r1;
            q *= r1;
        }
        char* h = a.H + i * a.ldh * ES;
        float ss = 0.f;
        for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
            float fx[V::N], fr[V::N], w[V::N];
            V::load(x + v * 16, fx);
            V::load(r + v * 16, fr);
            if (a.post_gamma) {
                V::load(a.post_gamma + v * 16, w);
#pragma unroll
                for (int k = 0; k < V::N; ++k) fx[k] *= w[k];
            }
            if (a.gate_kind == FOAK_GATE_CHANNEL || a.gate_kind == FOAK_GATE_FULL) {
                V::load(g + v * 16, w);
#pragma unroll
                for (int k = 0; k < V::N; ++k) fx[k] *= w[k];
            }
#pragma unroll
            for (int k = 0; k < V::N; ++k) {
                fr[k] = fmaf(q, fx[k], fr[k]);
                ss = fmaf(fr[k], fr[k], ss);
                row_h[v * V::N + k] = fr[k];
            }
            V::store(h + v * 16, fr);
        }
        if (a.gamma) {
            const float rstd = rsqrtf(block_sum(ss, red[1]) * inv_d + a.eps);
            if (threadIdx.x == 0 && a.rstd) a.rstd[i] = rstd;
            char* y = a.Y + i * a.ldy * ES;
            for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
                float w[V::N];
                V::load(a.gamma + v * 16, w);
#pragma unroll
                for (int k = 0; k < V::N; ++k) w[k] *= row_h[v * V::N + k] * rstd;
                V::store(y + v * 16, w);
            }
        }
        __syncthreads();  // red is free again
    }
}

// What a row's elements need of the row's sums: dh = dH + r gamma dY - k1 H, and with the norm after
// the block dX = r1 gp du - k2 X.
struct RowStats {
    float k1, k2;
};

template <int ES>
__device__ __forceinline__ const char* gate_row(const ResNormBwd& a, int64_t i) {
    return a.gate_kind == FOAK_GATE_CHANNEL ? a.gate : a.gate + i * a.ldg * ES;
}

template <int ES>
__device__ __forceinline__ float row_factor(const ResNormBwd& a, int64_t i) {
    return a.gate_kind == FOAK_GATE_ROW ? a.scale * Vec16<ES>::load1(gate_row<ES>(a, i)) : a.scale;
}

// The sums of each row, a CTA a row: m D = sum hh t; and, over w = u without s (and without the gate of a
// row), E = sum dh w = sum w (dH + r t) - r m sum w hh, which is the row gate's gradient without s, and
// s E (times the row's gate) the sum of xh gp du.
template <int ES>
__global__ void __launch_bounds__(256) resnorm_bwd_stats_kernel(const ResNormBwd a, RowStats* stats) {
    griddep_launch_dependents();  // programmatic dependent launch: no global access before the wait
    griddep_wait();
    using V = Vec16<ES>;
    __shared__ float red[3][32];
    const int nvec = static_cast<int>(a.D / V::N);
    const float inv_d = 1.f / static_cast<float>(a.D);
    const bool sums = a.post_gamma || (a.gate_kind == FOAK_GATE_ROW && a.dgate);
    const bool elem_gate = a.gate_kind == FOAK_GATE_CHANNEL || a.gate_kind == FOAK_GATE_FULL;
    for (int64_t i = blockIdx.x; i < a.N; i += gridDim.x) {
        const float r = a.dY ? a.rstd[i] : 0.f, r1 = a.post_gamma ? a.post_rstd[i] : 1.f;
        float s1 = 0.f, s2 = 0.f, s3 = 0.f;
        for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
            float t[V::N], hh[V::N], d[V::N], w[V::N];
#pragma unroll
            for (int k = 0; k < V::N; ++k) t[k] = hh[k] = d[k] = 0.f;
            if (a.dY) {
                V::load(a.dY + (i * a.lddy + v * V::N) * ES, t);
                V::load(a.gamma + v * 16, w);
                V::load(a.H + (i * a.ldh + v * V::N) * ES, hh);
#pragma unroll
                for (int k = 0; k < V::N; ++k) {
                    t[k] *= w[k];
                    hh[k] *= r;
                    s1 = fmaf(hh[k], t[k], s1);
                }
            }
            if (!sums) continue;
            if (a.dH) V::load(a.dH + (i * a.lddh + v * V::N) * ES, d);
            V::load(a.X + (i * a.ldx + v * V::N) * ES, w);
            if (a.post_gamma) {
                float gp[V::N];
                V::load(a.post_gamma + v * 16, gp);
#pragma unroll
                for (int k = 0; k < V::N; ++k) w[k] *= r1 * gp[k];
            }
            if (elem_gate) {
                float e[V::N];
                V::load(gate_row<ES>(a, i) + v * 16, e);
#pragma unroll
                for (int k = 0; k < V::N; ++k) w[k] *= e[k];
            }
#pragma unroll
            for (int k = 0; k < V::N; ++k) {
                s2 = fmaf(w[k], fmaf(r, t[k], d[k]), s2);
                s3 = fmaf(w[k], hh[k], s3);
            }
        }
        s1 = block_sum(s1, red[0]);
        if (sums) {
            s2 = block_sum(s2, red[1]);
            s3 = block_sum(s3, red[2]);
        }
        if (threadIdx.x == 0) {
            const float m = s1 * inv_d, E = s2 - r * m * s3;
            stats[i] = RowStats{r * r * m, r1 * r1 * inv_d * row_factor<ES>(a, i) * E};
            if (a.gate_kind == FOAK_GATE_ROW && a.dgate) reinterpret_cast<float*>(a.dgate)[i] = a.scale * E;
        }
        __syncthreads();  // red is free again
    }
}

// The gradients of a range of columns for a group of rows, and the group's part of the sums over the rows:
// part1 = sum dy hh;  part2 = sum dh xh (X without the norm after the block), times s e where e is one a row
// or an element.
template <int ES>
__global__ void __launch_bounds__(128) resnorm_bwd_cols_kernel(const ResNormBwd a, const RowStats* stats, float* part1,
                                                               float* part2) {
    griddep_launch_dependents();  // programmatic dependent launch: no global access before the wait
    griddep_wait();
    using V = Vec16<ES>;
    const int64_t v = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
    if (v * V::N >= a.D) return;
    float gm[V::N], gp[V::N], e[V::N], acc1[V::N], acc2[V::N];
#pragma unroll
    for (int k = 0; k < V::N; ++k) {
        gm[k] = 0.f;
        gp[k] = e[k] = 1.f;
        acc1[k] = acc2[k] = 0.f;
    }
    if (a.dY) V::load(a.gamma + v * 16, gm);
    if (a.post_gamma) V::load(a.post_gamma + v * 16, gp);
    if (a.gate_kind == FOAK_GATE_CHANNEL) V::load(a.gate + v * 16, e);
    const bool weighted = a.gate_kind == FOAK_GATE_ROW || a.gate_kind == FOAK_GATE_FULL;
    const int64_t col = v * V::N;
    for (int64_t i = blockIdx.y; i < a.N; i += gridDim.y) {
        const float r = a.dY ? a.rstd[i] : 0.f, r1 = a.post_gamma ? a.post_rstd[i] : 1.f, q = row_factor<ES>(a, i);
        const RowStats st = stats[i];
        float dh[V::N], x[V::N];
#pragma unroll
        for (int k = 0; k < V::N; ++k) dh[k] = x[k] = 0.f;
        if (a.dH) V::load(a.dH + (i * a.lddh + col) * ES, dh);
        if (a.X) V::load(a.X + (i * a.ldx + col) * ES, x);
        if (a.dY) {
            float dy[V::N], h[V::N];
            V::load(a.dY + (i * a.lddy + col) * ES, dy);
            V::load(a.H + (i * a.ldh + col) * ES, h);
#pragma unroll
            for (int k = 0; k < V::N; ++k) {
                acc1[k] = fmaf(dy[k], h[k] * r, acc1[k]);
                dh[k] += fmaf(r * gm[k], dy[k], -st.k1 * h[k]);
            }
        }
        if (a.gate_kind == FOAK_GATE_FULL) V::load(a.gate + (i * a.ldg + col) * ES, e);
        float dx[V::N], dg[V::N];
#pragma unroll
        for (int k = 0; k < V::N; ++k) {
            const float du = q * e[k] * dh[k], xh = x[k] * r1;
            acc2[k] = fmaf(weighted ? du : dh[k], xh, acc2[k]);
            dx[k] = a.post_gamma ? r1 * gp[k] * du - st.k2 * x[k] : du;
            dg[k] = q * dh[k] * (xh * gp[k]);
        }
        V::store(a.dR + (i * a.lddr + col) * ES, dh);
        if (a.dX) V::store(a.dX + (i * a.lddx + col) * ES, dx);
        if (a.gate_kind == FOAK_GATE_FULL && a.dgate) V::store(a.dgate + (i * a.lddg + col) * ES, dg);
    }
#pragma unroll
    for (int k = 0; k < V::N; ++k) {
        if (a.dgamma) part1[blockIdx.y * a.D + col + k] = acc1[k];
        if (part2) part2[blockIdx.y * a.D + col + k] = acc2[k];
    }
}

// The sums over the groups in a fixed order: 32 slices of 32 columns a CTA, each adding every 32nd group,
// then the slices in order.  blockIdx.y 0: dgamma; 1: the gate's and the post norm's from the same sums.
constexpr int kRedCols = 32, kRedSlices = 32, kRedMaxG = 512;
template <int ES>
__global__ void __launch_bounds__(kRedCols * kRedSlices)
    resnorm_reduce_kernel(const ResNormBwd a, const float* part1, const float* part2, int G) {
    griddep_launch_dependents();  // programmatic dependent launch: no global access before the wait
    griddep_wait();
    using V = Vec16<ES>;
    __shared__ float ss[kRedSlices][kRedCols];
    const bool second = blockIdx.y == 1 || !a.dgamma;
    const float* part = second ? part2 : part1;
    const int c = threadIdx.x % kRedCols, sl = threadIdx.x / kRedCols;
    const int64_t j = static_cast<int64_t>(blockIdx.x) * kRedCols + c;
    float s = 0.f;
    if (j < a.D) {
        float val[kRedMaxG / kRedSlices];
#pragma unroll
        for (int i = 0; i < kRedMaxG / kRedSlices; ++i) {
            const int g = sl + i * kRedSlices;
            val[i] = g < G ? part[static_cast<int64_t>(g) * a.D + j] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kRedMaxG / kRedSlices; ++i) s += val[i];
    }
    ss[sl][c] = s;
    __syncthreads();
    if (sl != 0 || j >= a.D) return;
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < kRedSlices; ++k) t += ss[k][c];
    if (!second) {
        a.dgamma[j] = t;
        return;
    }
    const bool channel = a.gate_kind == FOAK_GATE_CHANNEL;
    if (channel && a.dgate)
        reinterpret_cast<float*>(a.dgate)[j] = a.scale * t * (a.post_gamma ? V::load1(a.post_gamma + j * ES) : 1.f);
    if (a.dpost_gamma) {
        if (channel) t *= a.scale * V::load1(a.gate + j * ES);
        if (a.gate_kind == FOAK_GATE_NONE) t *= a.scale;
        a.dpost_gamma[j] = t;
    }
}

// Once per device: dynamic shared memory above 48 KB.
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, bool (&done)[64]) {
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    done[dev] = e == cudaSuccess;
    return e;
}

template <int ES>
cudaError_t fwd(const ResNormFwd& a, cudaStream_t s) {
    static bool done[64] = {};
    const cudaError_t e = allow_smem(resnorm_fwd_row_kernel<ES>, static_cast<int>(kResNormMaxD) * 4, done);
    if (e != cudaSuccess) return e;
    const int64_t nvec = a.D / (16 / ES);
    const int threads = nvec <= 256 ? static_cast<int>((nvec + 31) / 32 * 32) : nvec <= 1024 ? 256 : 512;
    const int grid = static_cast<int>(std::min<int64_t>(a.N, static_cast<int64_t>(device_sm_count()) * 8));
    return launch_dependent(resnorm_fwd_row_kernel<ES>, dim3(grid), dim3(threads), static_cast<size_t>(a.D) * 4, s, a);
}

template <int ES>
cudaError_t bwd(const ResNormBwd& a, void* workspace, cudaStream_t s) {
    const int groups = resnorm_groups(a.D);
    float* part1 = static_cast<float*>(workspace);
    float* part2 = part1 + static_cast<size_t>(groups) * a.D;
    RowStats* stats = reinterpret_cast<RowStats*>(part2 + static_cast<size_t>(groups) * a.D);
    const bool second = (a.gate_kind == FOAK_GATE_CHANNEL && a.dgate) || a.dpost_gamma;
    const int64_t nvec = a.D / (16 / ES);
    const int G = static_cast<int>(std::min<int64_t>(std::max<int64_t>(a.N, 1), 128));
    cudaError_t e = cudaSuccess;
    if (a.N > 0) {
        const int grid = static_cast<int>(std::min<int64_t>(a.N, static_cast<int64_t>(device_sm_count()) * 8));
        e = launch_dependent(resnorm_bwd_stats_kernel<ES>, dim3(grid), dim3(256), 0, s, a, stats);
        if (e != cudaSuccess) return e;
    }
    e = launch_dependent(resnorm_bwd_cols_kernel<ES>, dim3(static_cast<unsigned>((nvec + 127) / 128), G), dim3(128), 0,
                         s, a, static_cast<const RowStats*>(stats), part1, second ? part2 : nullptr);
    if (e != cudaSuccess || (!a.dgamma && !second)) return e;
    const dim3 rgrid(static_cast<unsigned>((a.D + kRedCols - 1) / kRedCols), a.dgamma && second ? 2 : 1);
    return launch_dependent(resnorm_reduce_kernel<ES>, rgrid, dim3(kRedCols * kRedSlices), 0, s, a,
                            static_cast<const float*>(part1), static_cast<const float*>(part2), G);
}

}  // namespace

cudaError_t launch_resnorm_fwd(int es, const ResNormFwd& a, cudaStream_t s) {
    if (a.N == 0) return cudaSuccess;
    return es == 2 ? fwd<2>(a, s) : fwd<4>(a, s);
}

cudaError_t launch_resnorm_bwd(int es, const ResNormBwd& a, void* workspace, cudaStream_t s) {
    return es == 2 ? bwd<2>(a, workspace, s) : bwd<4>(a, workspace, s);
}

}  // namespace foak
