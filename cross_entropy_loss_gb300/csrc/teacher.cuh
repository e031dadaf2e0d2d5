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
    alignas(16) int id[kTeacherMax];      // -1: no entry (also past K, up to a multiple of 4)
    alignas(16) float q[kTeacherMax];
    float lnq[kTeacherMax];
    float x[kTeacherMax];                 // the student's logit of the token (only where col_lo <= id < col_hi)
    alignas(16) int seen[2 * kTeacherMax];  // hash table of the ids
    float total;                          // sum of q
    bool repeated;                        // a token is listed more than once
};

// The row's targets, by a whole warp, which is in step afterwards.  Returns whether an id
// was V or more (such an entry, like one with a negative id, counts as absent).
// (Loops over shared memory: unrolled over a lane's eight entries in registers, the code
// crowds the streaming warps' out of the instruction cache.)
__device__ __forceinline__ bool teacher_row(const TeacherSrc& p, int64_t row, int64_t V, TeacherRow& out) {
    constexpr int PER = kTeacherMax / 32;
    const int lane = threadIdx.x & 31, K4 = (p.K + 3) / 4 * 4;
    const int32_t* ids = p.ids + row * p.ld;
    const float* logp = p.logp + row * p.ld;
    int id[PER];
    float t[PER];
    // all loads go out together
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int k = lane + 32 * j;
        id[j] = -1;
        t[j] = kNegInf;
        if (k < p.K) {
            id[j] = __ldg(ids + k);
            t[j] = __ldg(logp + k);
        }
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int k = lane + 32 * j;
        if (k < K4) {
            out.id[k] = id[j];
            out.lnq[k] = t[j];
        }
    }
#pragma unroll 1
    for (int j = lane; j < 2 * kTeacherMax / 4; j += 32) reinterpret_cast<int4*>(out.seen)[j] = make_int4(-1, -1, -1, -1);
    __syncwarp();
    bool bad = false, twice = false;
    float top = kNegInf;
#pragma unroll 1
    for (int k = lane; k < K4; k += 32) {
        const int i = out.id[k];
        bad |= i >= V;
        if (i < 0 || i >= V) {
            out.id[k] = -1;
            out.lnq[k] = kNegInf;
            continue;
        }
        // at most half of the table fills
        for (unsigned h = (static_cast<unsigned>(i) * 2654435761u) >> 23;; h = (h + 1) & (2 * kTeacherMax - 1)) {
            const int before = atomicCAS(out.seen + h, -1, i);
            twice |= before == i;
            if (before == -1 || before == i) break;
        }
        top = fmaxf(top, out.lnq[k]);
    }
    static_assert(2 * kTeacherMax == 1 << (32 - 23), "the hash takes the table's bits");
    __syncwarp();
    top = p.normalize ? warp_max(top) : 0.f;
    // q = e^t, or that over its sum; the sum is taken below the largest so that it cannot overflow
    float sum = 0.f;
#pragma unroll 1
    for (int k = lane; k < K4; k += 32) {
        const float v = out.lnq[k], q = v == kNegInf ? 0.f : expf(v - top);
        out.q[k] = q;
        sum += q;
    }
    sum = warp_sum(sum);
    const bool over = p.normalize && sum > 0.f;
    if (over) {
        const float ln_norm = top + logf(sum);
#pragma unroll 1
        for (int k = lane; k < K4; k += 32) {
            out.lnq[k] -= ln_norm;
            out.q[k] /= sum;  // the quotient, not e^(t - ln norm): its rounding stays relative to q
        }
    }
    twice = __any_sync(0xffffffffu, twice);
    if (lane == 0) {
        out.total = over ? 1.f : sum;
        out.repeated = twice;
    }
    bad = __any_sync(0xffffffffu, bad);
    __syncwarp();
    return bad;
}
// The student's logits of the listed tokens in [col_lo, col_hi), by a whole warp.
template <int ES>
__device__ __forceinline__ void teacher_gather(int K, const char* rowp, int64_t col_lo, int64_t col_hi, TeacherRow& out) {
#pragma unroll 4
    for (int k = threadIdx.x & 31; k < K; k += 32) {
        const int id = out.id[k];
        if (id >= col_lo && id < col_hi) out.x[k] = load_scalar<ES>(rowp + static_cast<int64_t>(id) * ES);
    }
    __syncwarp();
}

// A warp's corrections of a row's gradient in the columns [col_lo, col_hi): what the K
// listed tokens and the label y (-1: none; its logit x_y) take off the plain gradient
// `grad_at` of their logits.  A token listed twice gets the same value from each place.
template <int ES, typename F>
__device__ __forceinline__ void teacher_correct(const TeacherRow& t, int K, int64_t col_lo, int64_t col_hi, int64_t y,
                                                float x_y, float w1, float wt, char* drow, F&& grad_at) {
    const int lane = threadIdx.x & 31;
    bool listed = false;
#pragma unroll 1
    for (int k = lane; k < K; k += 32) {
        const int id = t.id[k];
        if (id < 0 || id < col_lo || id >= col_hi) continue;
        float mass = t.q[k];
        if (t.repeated) {
            mass = 0.f;
#pragma unroll 1
            for (int j = 0; j < K; ++j) mass += t.id[j] == id ? t.q[j] : 0.f;
        }
        float e = grad_at(t.x[k]) - wt * mass;
        if (id == y) {
            e -= w1;
            listed = true;
        }
        store_scalar<ES>(drow + static_cast<int64_t>(id) * ES, e);
    }
    listed = __any_sync(0xffffffffu, listed);
    if (lane == 0 && !listed && y >= col_lo && y < col_hi) store_scalar<ES>(drow + y * ES, grad_at(x_y) - w1);
}

}  // namespace foak
