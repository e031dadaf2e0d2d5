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
// Both directions are bound by memory: each operand is read and each result written once (fp32 sums in
// a fixed order: results are the same from run to run).
#include <algorithm>

#include "foak_ce.h"
#include "internal.h"
#include "launch_once.h"
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

constexpr int kVpt = 2;
constexpr int kRowThreads = 512;
constexpr int kMaxCluster = 8;
constexpr int kRingSmem = 208 * 1024;  // of an SM's CTAs together, 512 threads; beside it each CTA's sums
constexpr int kRingSmemMax = 224 * 1024;
constexpr size_t kSmSmem = 228 * 1024;

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// A 16-byte vector as element pairs.
template <int ES>
struct Pairs {
    static constexpr int N = 8 / ES;
    float2 p[N];
    __device__ __forceinline__ void unpack(const uint4& w) {
        if constexpr (ES == 2) {
            p[0] = make_float2(bf16_lo(w.x), bf16_hi(w.x));
            p[1] = make_float2(bf16_lo(w.y), bf16_hi(w.y));
            p[2] = make_float2(bf16_lo(w.z), bf16_hi(w.z));
            p[3] = make_float2(bf16_lo(w.w), bf16_hi(w.w));
        } else {
            p[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
            p[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
        }
    }
    __device__ __forceinline__ void store(char* dst) const {
        uint4 w;
        if constexpr (ES == 2)
            w = make_uint4(pack_bf16x2(p[0].x, p[0].y), pack_bf16x2(p[1].x, p[1].y), pack_bf16x2(p[2].x, p[2].y),
                           pack_bf16x2(p[3].x, p[3].y));
        else
            w = make_uint4(__float_as_uint(p[0].x), __float_as_uint(p[0].y), __float_as_uint(p[1].x),
                           __float_as_uint(p[1].y));
        *reinterpret_cast<uint4*>(dst) = w;
    }
    __device__ __forceinline__ void fill(float v) {
#pragma unroll
        for (int k = 0; k < N; ++k) p[k] = make_float2(v, v);
    }
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }


// ------------------------------------------------------------------ forward
// A CTA a row at a time, h kept in shared memory as floats (each thread's own vectors) between the sum of
// its squares and y; with the norm after the block X is read once more, from L1 or L2, for its own sum
// first.  The second sum is of h itself: expanding it into sums of R and X would cancel where the
// block takes the residual back.
//
// Bound by memory; what counts is how many rows an SM has under way, since a row waits for its loads and at
// its barriers.  So: 32 registers, two vectors a thread and operand, their loads one vector at a time, and
// grids of four times what is resident.  Measured (bf16, us): 8192 x 4096 41.0, 98% of the copy rate (one
// vector a thread 42.5, four 49.3; 64 registers and two vectors at a time 43.6; a ring of cp.async rows
// 44.8), with both norms 44.9 (ring 49.4, X and R kept in shared memory 53); 16384 x 1024 22.4; 3000 x 10240
// 39.3 and 2048 x 16384 43.6 (512 threads for wide rows 40.6 and 50.0, with 64 registers 47.2 and 45.2).
constexpr int kFwdThreads = 1024;

template <int ES, bool POST, bool FULL>
__global__ void __launch_bounds__(kFwdThreads, 2) resnorm_fwd_kernel(const __grid_constant__ ResNormFwd a) {
    griddep_launch_dependents();  // programmatic dependent launch: no global access before the wait
    griddep_wait();
    using P = Pairs<ES>;
    constexpr int EPV = 16 / ES, NP = P::N;
    extern __shared__ uint4 kept[];  // h: [4 / ES planes of 16 bytes][vectors]
    __shared__ float red[4][32];
    const int nvec = static_cast<int>(a.D / EPV), nt = blockDim.x;
    const float inv_d = 1.f / static_cast<float>(a.D);
    const bool channel = !FULL && a.gate_kind == FOAK_GATE_CHANNEL;
    auto squares = [](const uint4& w, float2 s) {
        P p;
        p.unpack(w);
#pragma unroll
        for (int k = 0; k < NP; ++k) s = __ffma2_rn(p.p[k], p.p[k], s);
        return s;
    };
    int buffer = 0;  // two rows in a row use different ones of `red`
    for (int64_t i = blockIdx.x; i < a.N; i += gridDim.x, buffer ^= 2) {
        const char* xr = a.X + i * a.ldx * ES;
        const char* rr = a.R + i * a.ldr * ES;
        const char* gr = channel ? a.gate : a.gate + i * a.ldg * ES;
        char* hr = a.H + i * a.ldh * ES;
        float q = a.scale;
        if (!FULL && a.gate_kind == FOAK_GATE_ROW) q *= Vec16<ES>::load1(gr);
        if constexpr (POST) {
            float2 sx = both(0.f);
            for (int v = threadIdx.x; v < nvec; v += nt) sx = squares(ld_global_v4(xr + v * 16), sx);
            const float r1 = rsqrtf(block_sum(sx.x + sx.y, red[buffer]) * inv_d + a.post_eps);
            if (threadIdx.x == 0 && a.post_rstd) a.post_rstd[i] = r1;
            q *= r1;
        }
        float2 s2 = both(0.f);
        for (int v = threadIdx.x; v < nvec; v += nt) {
            P x, h, w;
            x.unpack(ld_global_v4(xr + v * 16));
            h.unpack(ld_global_v4(rr + v * 16));
            if constexpr (POST) {
                w.unpack(ld_global_v4(a.post_gamma + v * 16));
#pragma unroll
                for (int k = 0; k < NP; ++k) x.p[k] = __fmul2_rn(x.p[k], w.p[k]);
            }
            if (FULL || channel) {
                w.unpack(ld_global_v4(gr + v * 16));
#pragma unroll
                for (int k = 0; k < NP; ++k) x.p[k] = __fmul2_rn(x.p[k], w.p[k]);
            }
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                h.p[k] = __ffma2_rn(both(q), x.p[k], h.p[k]);
                s2 = __ffma2_rn(h.p[k], h.p[k], s2);
            }
            h.store(hr + v * 16);
            if (a.gamma) {
#pragma unroll
                for (int k = 0; k < NP; k += 2)
                    kept[k / 2 * nvec + v] = make_uint4(__float_as_uint(h.p[k].x), __float_as_uint(h.p[k].y),
                                                        __float_as_uint(h.p[k + 1].x), __float_as_uint(h.p[k + 1].y));
            }
        }
        float rstd = 0.f;
        if (a.gamma) {
            rstd = rsqrtf(block_sum(s2.x + s2.y, red[buffer + 1]) * inv_d + a.eps);
            if (threadIdx.x == 0 && a.rstd) a.rstd[i] = rstd;
        }
        if (a.gamma) {
            char* yr = a.Y + i * a.ldy * ES;
            for (int v = threadIdx.x; v < nvec; v += nt) {
                P w;
                w.unpack(ld_global_v4(a.gamma + v * 16));
#pragma unroll
                for (int k = 0; k < NP; k += 2) {
                    const uint4 f = kept[k / 2 * nvec + v];
                    const float2 lo = make_float2(__uint_as_float(f.x), __uint_as_float(f.y));
                    const float2 hi = make_float2(__uint_as_float(f.z), __uint_as_float(f.w));
                    w.p[k] = __fmul2_rn(__fmul2_rn(lo, both(rstd)), w.p[k]);
                    w.p[k + 1] = __fmul2_rn(__fmul2_rn(hi, both(rstd)), w.p[k + 1]);
                }
                w.store(yr + v * 16);
            }
        }
    }
}

// ------------------------------------------------------------------ backward, any rows
// Sums first, then the columns: for row strides or counts past 32 bits, and for a full gate whose gradient nobody
// wants (bf16 8192 x 4096 163 us, where the one-pass kernel takes 92 with that gradient; 13534 x 560 198 and 26).
// What a row's elements need of the row's sums (RowStats): dh = dH + r gamma dY - k1 H, and with the norm after the
// block dX = r1 gp du - k2 X.
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

// ------------------------------------------------------------------ backward, one pass
// Rows in slices of at most 1024 vectors, a CTA each, those of a row one cluster; a cluster takes a range of
// rows.  Thread v owns vectors v and v + threads of its slice, so the sums over the rows stay in registers
// until the end.  Every thread copies its own vectors of a row's operands into a ring of shared
// memory, stages - 1 rows ahead (cp.async: a hardware wait, no spin), takes its part of what the row needs,
// meets the others at one barrier a row and reads its vectors again for the results.  The row's sums have r
// and r1 factored out (w = gp e x, e the gate of a channel or an element; q = s, times the gate of a row):
//     S1 = sum h gamma dy,   S2 = sum w (dH + r gamma dy),   S3 = sum w h,   k1 = r^3 S1 / D
//     dh = dH + r gamma dy - k1 h,   E = sum dh w r1 = r1 (S2 - k1 S3),   k2 = r1^2 q E / D
//     dX = r1 q gp e dh - k2 x
// Arithmetic on pairs (two-wide FP32).
//
// Bound by memory and, in bf16, by how many instructions 16 warps an SM get out (half of the issue slots).  bf16,
// us: 8192 x 4096 60 (0.83 of the copy rate; the reduce 4 to 6 of them), both norms and a channel gate 73; 4096 x
// 8192 59 (256 threads and clusters of two 70); 2048 x 16384 64 (waiting at the barrier for the row's sums, not
// with the next row's sums in between, 87); 8192 x 4096 reading each operand twice, sums first, 139.  An element's
// intermediate results kept across the barrier spill: 86 against 71 with both norms.
// The warp's sums of four values with six shuffles: lanes 8 v .. 8 v + 7 get value v.
__device__ __forceinline__ float warp_sum4(float a, float b, float c, float d, int lane) {
    const bool hi = lane & 16, odd = lane & 8;
    const float x = (hi ? c : a) + __shfl_xor_sync(0xffffffffu, hi ? a : c, 16);
    const float y = (hi ? d : b) + __shfl_xor_sync(0xffffffffu, hi ? b : d, 16);
    float z = (odd ? y : x) + __shfl_xor_sync(0xffffffffu, odd ? x : y, 8);
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
    return z;
}

// Stages of the ring, of `operands` each: as many as leave room for 512 threads an SM.
constexpr int ring_stages(int operands) {
    const int n = kRingSmem / kRowThreads / (operands * kVpt * 16);
    return n < 4 ? n : 4;
}
static_assert(ring_stages(3) == 4 && ring_stages(4) == 3 && ring_stages(5) == 2, "two stages or more");

struct BwdSplit {
    int cluster;             // CTAs a row
    int slice;               // vectors of a CTA's slice
    uint32_t in[5], out[3];  // bytes from row to row of dY, H, dH, X, gate; dR, dX, dgate
};

// SUMS: S2 and S3 are wanted (the norm after the block, or the gradient of a row's gate).
template <int ES, bool POST, bool FULL, bool HASX, bool SUMS>
__global__ void __launch_bounds__(kRowThreads, 1)
    resnorm_bwd_ring_kernel(const __grid_constant__ ResNormBwd a, const BwdSplit sp, float* __restrict__ part1,
                            float* __restrict__ part2) {
    griddep_launch_dependents();  // programmatic dependent launch: no global access before the wait
    using P = Pairs<ES>;
    constexpr int EPV = 16 / ES, NP = P::N, NS = 3 + HASX + FULL, NSUM = SUMS ? 4 : 1, kStages = ring_stages(NS);
    extern __shared__ uint4 ring[];  // [stages][NS][kVpt][threads], then the rows' sums: [2][warps of the cluster][NSUM]
    const int v = threadIdx.x, lane = v & 31, warp = v >> 5, nt = blockDim.x, warps = nt >> 5;
    const int C = sp.cluster, rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int64_t cid = C > 1 ? static_cast<int64_t>(blockIdx.x) / C : blockIdx.x, clusters = gridDim.x / C;
    bool act[kVpt];
    int off[kVpt];  // bytes from the row's begin
#pragma unroll
    for (int j = 0; j < kVpt; ++j) {
        const int at = v + j * nt;
        off[j] = (rank * sp.slice + at) * 16;
        act[j] = at < sp.slice && off[j] < static_cast<int>(a.D) * ES;
    }
    const int64_t r_begin = a.N * cid / clusters;
    const int rows = static_cast<int>(a.N * (cid + 1) / clusters - r_begin);
    const float inv_d = 1.f / static_cast<float>(a.D);
    const int plane = kVpt * nt;  // vectors of an operand
    float* red = reinterpret_cast<float*>(ring + kStages * NS * plane);
    // An operand that is not there reads as zeros, and so does a vector past the slice's end: the sums below
    // go through all of a thread's vectors without a branch.
#pragma unroll
    for (int j = 0; j < kVpt; ++j) {
        for (int i = 0; i < kStages * NS; ++i) {
            const int operand = i % NS;
            if (!act[j] || (operand < 2 && !a.dY) || (operand == 2 && !a.dH))
                ring[i * plane + j * nt + v] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    if (C > 1) cluster_sync();  // nobody writes into a CTA that has not begun
    griddep_wait();
    uint32_t next = static_cast<uint32_t>(r_begin);  // the row to copy
    const uint32_t last = next + rows;
    // its copies into stage s, one group a row (empty past the last, so that the count stays in step)
    auto issue = [&](int s) {
        if (next < last) {
            uint4* to = ring + s * (NS * plane) + v;
            auto copy = [&](int i, const char* base, uint32_t stride) {
                const char* p = base + static_cast<uint64_t>(next) * stride;
#pragma unroll
                for (int j = 0; j < kVpt; ++j)
                    if (act[j]) cp_async16(to + i * plane + j * nt, p + off[j]);
            };
            if (a.dY) {
                copy(0, a.dY, sp.in[0]);
                copy(1, a.H, sp.in[1]);
            }
            if (a.dH) copy(2, a.dH, sp.in[2]);
            if constexpr (HASX) copy(3, a.X, sp.in[3]);
            if constexpr (FULL) copy(NS - 1, a.gate, sp.in[4]);
            ++next;
        }
        cp_async_commit();
    };
    for (int s = 0; s < kStages - 1; ++s) issue(s);
    P gm[kVpt], pe[kVpt], acc1[kVpt], acc2[kVpt];
#pragma unroll
    for (int j = 0; j < kVpt; ++j) {
        gm[j].fill(0.f);
        pe[j].fill(1.f);
        acc1[j].fill(0.f);
        acc2[j].fill(0.f);
        if (!act[j]) continue;
        if (a.dY) gm[j].unpack(ld_global_v4(a.gamma + off[j]));
        if constexpr (POST) pe[j].unpack(ld_global_v4(a.post_gamma + off[j]));
        if (!FULL && a.gate_kind == FOAK_GATE_CHANNEL) {
            P e;
            e.unpack(ld_global_v4(a.gate + off[j]));
#pragma unroll
            for (int k = 0; k < NP; ++k) pe[j].p[k] = __fmul2_rn(pe[j].p[k], e.p[k]);
        }
    }
    const bool row_gate = !FULL && a.gate_kind == FOAK_GATE_ROW;
    struct Scalars {
        float r, r1, q;
    };
    auto scalars = [&](int n) {
        Scalars c = {0.f, 1.f, a.scale};
        if (n < rows) {
            const int64_t row = r_begin + n;
            if (a.dY) c.r = a.rstd[row];
            if constexpr (POST) c.r1 = a.post_rstd[row];
            if (row_gate) c.q = row_factor<ES>(a, row);
        }
        return c;
    };
    // the warp's part of row n's sums, from the stage that holds it
    auto sums = [&](const uint4* slot, float r) {
        float2 s1 = both(0.f), s2 = both(0.f), s3 = both(0.f);
        const float2 rr = both(r);
#pragma unroll
        for (int j = 0; j < kVpt; ++j) {
            P dy, h, d, w;
            dy.unpack(slot[j * nt]);
            h.unpack(slot[plane + j * nt]);
            if constexpr (SUMS) {
                d.unpack(slot[2 * plane + j * nt]);
                w.unpack(slot[3 * plane + j * nt]);
                if constexpr (FULL) {
                    P e;
                    e.unpack(slot[(NS - 1) * plane + j * nt]);
#pragma unroll
                    for (int k = 0; k < NP; ++k) w.p[k] = __fmul2_rn(w.p[k], e.p[k]);
                }
            }
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const float2 t = __fmul2_rn(gm[j].p[k], dy.p[k]);
                s1 = __ffma2_rn(h.p[k], t, s1);
                if constexpr (SUMS) {
                    w.p[k] = __fmul2_rn(w.p[k], pe[j].p[k]);
                    s2 = __ffma2_rn(w.p[k], __ffma2_rn(rr, t, d.p[k]), s2);
                    s3 = __ffma2_rn(w.p[k], h.p[k], s3);
                }
            }
        }
        if constexpr (SUMS) return warp_sum4(s1.x + s1.y, s2.x + s2.y, s3.x + s3.y, 0.f, lane);
        else return warp_sum(s1.x + s1.y);
    };
    const int entries = C * warps;
    // To every CTA of the row, and arrive at its barrier.  The buffer's last readers, two rows ago, have arrived at
    // the barrier of the row before since, which this thread has passed.
    auto post = [&](int n, float z) {
        if (SUMS ? (lane & 7) == 0 : lane == 0) {
            float* mine = red + ((n & 1) * entries + rank * warps + warp) * NSUM + (SUMS ? lane >> 3 : 0);
            if (C == 1) *mine = z;
            else
                for (int c = 0; c < C; ++c) st_cluster_f32(mapa_u32(mine, c), z);
        }
        cluster_arrive_release();
    };
    // The next row's sums are taken between this one's arrival at its barrier and the wait there, where the ring
    // holds three rows or more; two rows of five operands are taken one after the other.
    constexpr bool kAhead = !FULL;
    int stage = 0;
    const auto slot_of = [&](int s) { return ring + s * (NS * plane) + v; };
    Scalars now = scalars(0), next_row = scalars(1);
    if constexpr (kAhead) {
        cp_async_wait<kStages - 2>();  // this thread's copies of the first row have landed
        if (rows > 0) post(0, sums(slot_of(0), now.r));
    }
    for (int n = 0; n < rows; ++n) {
        const Scalars ahead = scalars(n + 2);
        const float r = now.r, r1 = now.r1, q = now.q;
        const uint4* slot = slot_of(stage);
        const int free_stage = stage == 0 ? kStages - 1 : stage - 1;  // the row before's
        stage = stage + 1 == kStages ? 0 : stage + 1;
        issue(free_stage);
        cp_async_wait<kStages - (kAhead ? 2 : 1)>();
        float z_next = 0.f;
        if constexpr (kAhead) {
            if (n + 1 < rows) z_next = sums(slot_of(stage), next_row.r);
        } else post(n, sums(slot, r));
        cluster_wait_acquire();
        float S1, S2 = 0.f, S3 = 0.f, z = 0.f;
        const float* total = red + (n & 1) * entries * NSUM;
        if constexpr (SUMS) {
            for (int e = lane & 7; e < entries; e += 8) z += total[e * NSUM + (lane >> 3)];
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
            S1 = __shfl_sync(0xffffffffu, z, 0);
            S2 = __shfl_sync(0xffffffffu, z, 8);
            S3 = __shfl_sync(0xffffffffu, z, 16);
        } else {
            for (int e = lane; e < entries; e += 32) z += total[e];
            S1 = warp_sum(z);
        }
        if (kAhead && n + 1 < rows) post(n + 1, z_next);
        now = next_row;
        next_row = ahead;
        const float2 rr = both(r);
        const float k1 = r * r * (r * S1 * inv_d);
        float k2 = 0.f;
        if constexpr (SUMS) {
            const float E = r1 * (S2 - k1 * S3);
            k2 = r1 * r1 * (q * E * inv_d);
            if (row_gate && a.dgate && rank == 0 && v == 0) reinterpret_cast<float*>(a.dgate)[r_begin + n] = a.scale * E;
        }
        // dX = (r1 q) (gp e dh) - k2 x;  the sums over the rows take dh xh, weighted by a row's or an element's s e
        const uint64_t row = static_cast<uint32_t>(r_begin) + static_cast<uint32_t>(n);
        const float2 nk1 = both(-k1), nk2 = both(-k2), c = both(r1 * q), xw = both(FULL || row_gate ? r1 * q : r1);
#pragma unroll
        for (int j = 0; j < kVpt; ++j) {
            P dy, h, u, x, e, o;
            dy.unpack(slot[j * nt]);
            h.unpack(slot[plane + j * nt]);
            u.unpack(slot[2 * plane + j * nt]);
            if constexpr (POST || (HASX && (FULL || !SUMS))) x.unpack(slot[3 * plane + j * nt]);
            if constexpr (FULL) e.unpack(slot[(NS - 1) * plane + j * nt]);
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const float2 rdy = __fmul2_rn(rr, dy.p[k]);
                acc1[j].p[k] = __ffma2_rn(rdy, h.p[k], acc1[j].p[k]);
                const float2 d = __ffma2_rn(nk1, h.p[k], __ffma2_rn(gm[j].p[k], rdy, u.p[k]));
                u.p[k] = d;
                float2 g = pe[j].p[k];  // gp e
                if constexpr (FULL) {
                    const float2 dx = __fmul2_rn(d, __fmul2_rn(x.p[k], xw));  // s dh xh
                    if constexpr (POST) acc2[j].p[k] = __ffma2_rn(dx, e.p[k], acc2[j].p[k]);
                    if constexpr (POST) g = __fmul2_rn(g, e.p[k]);
                    else g = e.p[k];
                    e.p[k] = POST ? __fmul2_rn(dx, pe[j].p[k]) : dx;  // the gate's gradient
                } else if constexpr (POST) {
                    acc2[j].p[k] = __ffma2_rn(d, __fmul2_rn(x.p[k], xw), acc2[j].p[k]);
                } else if constexpr (HASX && !SUMS) {  // a channel's gate
                    acc2[j].p[k] = __ffma2_rn(d, x.p[k], acc2[j].p[k]);
                }
                if constexpr (POST) o.p[k] = __ffma2_rn(g, __fmul2_rn(c, d), __fmul2_rn(nk2, x.p[k]));
                else o.p[k] = __fmul2_rn(g, __fmul2_rn(c, d));
            }
            if (act[j]) {
                u.store(a.dR + row * sp.out[0] + off[j]);
                if (a.dX) o.store(a.dX + row * sp.out[1] + off[j]);
                if constexpr (FULL)
                    if (a.dgate) e.store(a.dgate + row * sp.out[2] + off[j]);
            }
        }
    }
    cp_async_wait<0>();  // no copy outlives the CTA (the trailing groups are empty)
#pragma unroll
    for (int j = 0; j < kVpt; ++j) {
        if (!act[j]) continue;
        const int64_t at = cid * a.D + off[j] / ES;
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            if (a.dgamma) *reinterpret_cast<float2*>(part1 + at + 2 * k) = acc1[j].p[k];
            if (HASX && part2) *reinterpret_cast<float2*>(part2 + at + 2 * k) = acc2[j].p[k];
        }
    }
}

// The sums over the groups in a fixed order: a CTA has 32 columns, its warps a slice of the groups each, whose sums the
// first warp adds in order.  blockIdx.y 0: dgamma; 1: the gate's and the post norm's from the same sums.  Bound by the
// latency of a round or two of loads from L2: as many warps as leave each about ten groups (76 groups of
// 2 x 16384 columns 10.2 us with 32 warps, 6.3 with 8; 304 of 2 x 4096 5.5 with 32, 6.3 with 16).  CTAs of 8 columns,
// or clusters over the groups, take 1 to 9 us longer.
constexpr int kRedCols = 32, kRedMaxWarps = 32;
template <int ES, int BATCH>
__global__ void __launch_bounds__(kRedCols * kRedMaxWarps)
    resnorm_reduce_kernel(const __grid_constant__ ResNormBwd a, const float* part1, const float* part2, int G) {
    griddep_launch_dependents();  // programmatic dependent launch: no global access before the wait
    griddep_wait();
    using V = Vec16<ES>;
    __shared__ float ss[kRedMaxWarps][kRedCols];
    const bool second = blockIdx.y == 1 || !a.dgamma;
    const float* part = second ? part2 : part1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t j = static_cast<int64_t>(blockIdx.x) * kRedCols + lane;
    float s = 0.f;
    if (j < a.D) {
        for (int g0 = warp; g0 < G; g0 += BATCH * warps) {  // a batch's loads go out together
            float val[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int g = g0 + i * warps;
                val[i] = g < G ? part[static_cast<int64_t>(g) * a.D + j] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) s += val[i];
        }
    }
    ss[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || j >= a.D) return;
    float t = 0.f;
    for (int k = 0; k < warps; k += 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) t += ss[k + i][lane];
    }
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

// The kernel on `clusters` clusters, as a programmatic dependent of the work before it.
template <typename... KA, typename... A>
cudaError_t launch_clusters(void (*kernel)(KA...), int64_t clusters, int cluster, int threads, size_t smem, cudaStream_t s,
                            A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * cluster));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

// How a row of nvec vectors is cut: CTAs, vectors of a CTA, its threads.
struct Slices {
    int cluster, slice, threads;
};

Slices slices_of(int64_t nvec) {
    Slices c = {1, 0, 0};
    while ((nvec + c.cluster - 1) / c.cluster > kVpt * kRowThreads) c.cluster *= 2;
    c.slice = static_cast<int>((nvec + c.cluster - 1) / c.cluster);
    c.threads = ((c.slice + kVpt - 1) / kVpt + 31) / 32 * 32;
    return c;
}

template <int ES, bool POST, bool FULL>
cudaError_t launch_fwd(const ResNormFwd& a, int threads, cudaStream_t s) {
    static SmemOnce limit;
    static ResidentOnce resident;
    const auto kernel = resnorm_fwd_kernel<ES, POST, FULL>;
    const size_t smem = a.gamma ? static_cast<size_t>(a.D) * 4 : 0;
    int ctas = 0;
    cudaError_t e = limit.allow(kernel, static_cast<int>(kResNormMaxD) * 4);
    if (e == cudaSuccess) e = resident.count(kernel, 1, threads, 0, &ctas);
    if (e != cudaSuccess) return e;
    // as many as the registers and threads allow, and the rows' shared memory
    const int64_t room = static_cast<int64_t>(kSmSmem / (smem + 2048)) * device_sm_count();
    const int64_t grid = std::min<int64_t>(a.N, std::min<int64_t>(ctas, room) * 4);
    return launch_clusters(kernel, grid, 1, threads, smem, s, a);
}

template <int ES>
cudaError_t fwd(const ResNormFwd& a, cudaStream_t s) {
    const bool full = a.gate_kind == FOAK_GATE_FULL;
    const int64_t nvec = a.D / (16 / ES);
    // Two vectors a thread; one where the rows do not fill the GPU (1 row of 4096 bf16 1.8 us against 2.2, 300 rows
    // 3.0 against 4.5).  Of fp32 rows with a norm after the block, which come by three times and keep half as much in
    // shared memory, four where that leaves CTAs of 256 to 512 threads (1537 x 5000 27.2 us against 29.4, 1500 x 7168
    // 35.7 against 38.7; near the ends 5482 x 4104 58.6 against 71.5, 2749 x 8184 59.5 against 67.1; bf16 of 2048
    // vectors 57.9 against 52.1).  Beyond either end four is faster as well where it was tried: 6250 x 3600 57.8
    // against 64.8, 2197 x 10240 56.4 against 63.9.
    const bool small = a.N <= 2 * static_cast<int64_t>(device_sm_count());
    const bool four = ES == 4 && a.post_gamma && nvec > 1024 && nvec < 2048;
    const int64_t each = small ? 1 : four ? 4 : 2;
    const int threads = static_cast<int>(std::min<int64_t>(((nvec + each - 1) / each + 31) / 32 * 32, kFwdThreads));
    if (a.post_gamma) return full ? launch_fwd<ES, true, true>(a, threads, s) : launch_fwd<ES, true, false>(a, threads, s);
    return full ? launch_fwd<ES, false, true>(a, threads, s) : launch_fwd<ES, false, false>(a, threads, s);
}

template <int ES, bool POST, bool FULL, bool HASX, bool SUMS>
cudaError_t launch_ring(const ResNormBwd& a, const BwdSplit& sp, int threads, float* part1, float* part2, int* groups,
                        cudaStream_t s) {
    const auto kernel = resnorm_bwd_ring_kernel<ES, POST, FULL, HASX, SUMS>;
    const size_t smem = static_cast<size_t>(ring_stages(3 + HASX + FULL)) * (3 + HASX + FULL) * kVpt * threads * 16 +
                        static_cast<size_t>(sp.cluster) * (threads / 32) * (SUMS ? 32 : 8);
    static SmemOnce limit;
    static ResidentOnce resident;
    int clusters = 0;
    cudaError_t e = limit.allow(kernel, kRingSmemMax);
    if (e == cudaSuccess) e = resident.count(kernel, sp.cluster, threads, smem, &clusters);
    if (e != cudaSuccess) return e;
    const int64_t G = std::min<int64_t>({a.N, clusters, resnorm_groups(a.N, a.D)});
    *groups = static_cast<int>(G);
    return launch_clusters(kernel, G, sp.cluster, threads, smem, s, a, sp, part1, part2);
}

template <int ES>
uint32_t bytes_of(int64_t ld) {
    return static_cast<uint32_t>(ld * ES);
}

template <int ES, bool POST, bool FULL, bool HASX, bool SUMS>
cudaError_t ring(const ResNormBwd& a, float* part1, float* part2, int* groups, cudaStream_t s) {
    const Slices c = slices_of(a.D / (16 / ES));
    const BwdSplit sp = {c.cluster, c.slice,
                         {bytes_of<ES>(a.lddy), bytes_of<ES>(a.ldh), bytes_of<ES>(a.lddh), bytes_of<ES>(a.ldx), bytes_of<ES>(a.ldg)},
                         {bytes_of<ES>(a.lddr), bytes_of<ES>(a.lddx), bytes_of<ES>(a.lddg)}};
    return launch_ring<ES, POST, FULL, HASX, SUMS>(a, sp, c.threads, part1, part2, groups, s);
}

// The sums over no rows.  No operand is read: nothing says that there are any.
cudaError_t bwd_of_no_rows(const ResNormBwd& a, cudaStream_t s) {
    const auto zero = [&](void* sums) {
        return sums ? cudaMemsetAsync(sums, 0, static_cast<size_t>(a.D) * sizeof(float), s) : cudaSuccess;
    };
    cudaError_t e = zero(a.dgamma);
    if (e == cudaSuccess) e = zero(a.dpost_gamma);
    if (e == cudaSuccess && a.gate_kind == FOAK_GATE_CHANNEL) e = zero(a.dgate);
    return e;
}

template <int ES>
cudaError_t bwd(const ResNormBwd& a, void* workspace, cudaStream_t s) {
    const int groups = resnorm_groups(a.N, a.D);
    float* part1 = static_cast<float*>(workspace);
    float* part2 = part1 + static_cast<size_t>(groups) * a.D;
    RowStats* stats = reinterpret_cast<RowStats*>(part2 + static_cast<size_t>(groups) * a.D);
    const bool second = (a.gate_kind == FOAK_GATE_CHANNEL && a.dgate) || a.dpost_gamma;
    const bool full = a.gate_kind == FOAK_GATE_FULL, row_grad = a.gate_kind == FOAK_GATE_ROW && a.dgate;
    const int64_t nvec = a.D / (16 / ES);
    int G = std::min(groups, kResNormColsGroups);
    cudaError_t e = cudaSuccess;
    // rows and row strides of 32 bits
    const int64_t ld = std::max({a.lddy, a.lddh, a.ldh, a.ldx, a.ldg, a.lddr, a.lddx, a.lddg});
    const bool one_pass = a.N < (1ll << 31) && ld * ES < (1ll << 32) && (a.X || !full);
    static_assert(kResNormMaxD / (16 / ES) <= kMaxCluster * kVpt * kRowThreads, "a row fits a cluster");
    if (one_pass) {
        float* p2 = second ? part2 : nullptr;
        if (a.post_gamma)
            e = full ? ring<ES, true, true, true, true>(a, part1, p2, &G, s) : ring<ES, true, false, true, true>(a, part1, p2, &G, s);
        else if (!a.X) e = ring<ES, false, false, false, false>(a, part1, p2, &G, s);
        else if (full) e = ring<ES, false, true, true, false>(a, part1, p2, &G, s);
        else e = row_grad ? ring<ES, false, false, true, true>(a, part1, p2, &G, s) : ring<ES, false, false, true, false>(a, part1, p2, &G, s);
        if (e != cudaSuccess) return e;
    } else {
        const int grid = static_cast<int>(std::min<int64_t>(a.N, static_cast<int64_t>(device_sm_count()) * 8));
        e = launch_dependent(resnorm_bwd_stats_kernel<ES>, dim3(grid), dim3(256), 0, s, a, stats);
        if (e != cudaSuccess) return e;
        e = launch_dependent(resnorm_bwd_cols_kernel<ES>, dim3(static_cast<unsigned>((nvec + 127) / 128), G), dim3(128), 0,
                             s, a, static_cast<const RowStats*>(stats), part1, second ? part2 : nullptr);
    }
    if (e != cudaSuccess || (!a.dgamma && !second)) return e;
    const dim3 rgrid(static_cast<unsigned>((a.D + kRedCols - 1) / kRedCols), a.dgamma && second ? 2 : 1);
    const int warps = G >= 256 ? kRedMaxWarps : G >= 128 ? kRedMaxWarps / 2 : kRedMaxWarps / 4;
    const auto reduce = G <= 10 * warps ? resnorm_reduce_kernel<ES, 10> : resnorm_reduce_kernel<ES, 20>;
    return launch_dependent(reduce, rgrid, dim3(32 * warps), 0, s, a, static_cast<const float*>(part1),
                            static_cast<const float*>(part2), G);
}

}  // namespace

cudaError_t launch_resnorm_fwd(int es, const ResNormFwd& a, cudaStream_t s) {
    if (a.N == 0) return cudaSuccess;
    return es == 2 ? fwd<2>(a, s) : fwd<4>(a, s);
}

cudaError_t launch_resnorm_bwd(int es, const ResNormBwd& a, void* workspace, cudaStream_t s) {
    if (a.N == 0) return bwd_of_no_rows(a, s);
    return es == 2 ? bwd<2>(a, workspace, s) : bwd<4>(a, workspace, s);
}

}  // namespace foak
