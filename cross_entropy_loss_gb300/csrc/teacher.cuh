// A teacher's top tokens of one row in shared memory: ids, probabilities and their
// logarithms, prepared by one warp.  Shared by the distillation kernels.
#pragma once

#include "common.cuh"
#include "row_common.cuh"

namespace foak {

constexpr int kTeacherMax = 256;

struct TeacherSrc {
    const int32_t* ids;  // [N][ld]
    const float* logp;   // [N][ld]
    int64_t ld;
    int K;
    bool normalize;
};

struct TeacherRow {
    alignas(16) int id[kTeacherMax];   // -1: no entry (also past K, up to a multiple of 4)
    alignas(16) float q[kTeacherMax];
    float lnq[kTeacherMax];
    float x[kTeacherMax];    // the student's logit of the token (only where col_lo <= id < col_hi)
    float total;             // sum of q
};

// Filled by a whole warp; the caller synchronises.  Returns whether an id was V or more
// (such an entry, like one with a negative id, counts as absent).  The student's logits
// are fetched for the ids in [col_lo, col_hi).
template <int ES>
__device__ __forceinline__ bool teacher_row(const TeacherSrc& p, int64_t row, int64_t V, const char* rowp,
                                            int64_t col_lo, int64_t col_hi, TeacherRow& out) {
    constexpr int PER = kTeacherMax / 32;
    const int lane = threadIdx.x & 31;
    float t[PER];
    bool bad = false;
    float top = kNegInf;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int k = lane + 32 * j;
        t[j] = kNegInf;
        if (k < p.K) {
            const int id = __ldg(p.ids + row * p.ld + k);
            const float v = __ldg(p.logp + row * p.ld + k);
            bad |= id >= V;
            const bool there = id >= 0 && id < V;
            out.id[k] = there ? id : -1;
            if (there) t[j] = v;
            if (there && id >= col_lo && id < col_hi) out.x[k] = load_scalar<ES>(rowp + static_cast<int64_t>(id) * ES);
        }
        if (k >= p.K && k < (p.K + 3) / 4 * 4) {
            out.id[k] = -1;
            out.q[k] = 0.f;
        }
        top = fmaxf(top, t[j]);
    }
    top = warp_max(top);
    // q = e^t, or that over its sum; the sum is taken below the largest so that it cannot overflow
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < PER; ++j)
        if (32 * j < p.K) sum += t[j] == kNegInf ? 0.f : expf(p.normalize ? t[j] - top : t[j]);
    sum = warp_sum(sum);
    const float ln_norm = p.normalize && sum > 0.f ? top + logf(sum) : 0.f;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int k = lane + 32 * j;
        if (k < p.K) {
            const float l = t[j] - ln_norm;
            out.lnq[k] = l;
            // the quotient, not e^(t - ln norm): its rounding stays relative to q
            out.q[k] = t[j] == kNegInf ? 0.f : (p.normalize ? expf(t[j] - top) / sum : expf(t[j]));
        }
    }
    if (lane == 0) out.total = p.normalize && sum > 0.f ? 1.f : sum;
    return __any_sync(0xffffffffu, bad);
}

// Sums of q over the entries with each of these ids (an id may be listed more than once).
template <int N>
__device__ __forceinline__ void teacher_mass(const TeacherRow& t, int K, const int (&id)[N], float (&mass)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n) mass[n] = 0.f;
    for (int k = 0; k < K; k += 4) {
        const int4 i = *reinterpret_cast<const int4*>(t.id + k);
        const float4 q = *reinterpret_cast<const float4*>(t.q + k);
#pragma unroll
        for (int n = 0; n < N; ++n)
            mass[n] += ((i.x == id[n] ? q.x : 0.f) + (i.y == id[n] ? q.y : 0.f)) +
                       ((i.z == id[n] ? q.z : 0.f) + (i.w == id[n] ? q.w : 0.f));
    }
}

}  // namespace foak
