// Arguments of the residual norms' launches (residual_norm.cu), checked by capi.cu.
// Strides are in elements; kinds of gate as FOAK_GATE_* of foak_ce.h.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace foak {

struct ResNormFwd {
    const char* X;
    const char* R;
    const char* gate;  // null: none
    const char* post_gamma;  // null: no norm after the block
    const char* gamma;  // null: H alone
    char* H;
    char* Y;
    float* post_rstd;
    float* rstd;
    int64_t ldx, ldr, ldg, ldh, ldy, N, D;
    int gate_kind;
    float scale, post_eps, eps;
};

struct ResNormBwd {
    const char* dY;  // null: the norm before the next block has no gradient
    const char* dH;  // null: none along the residual stream
    const char* H;
    const char* X;  // null where neither the norm after the block nor the gate's gradient needs it
    const char* gate;
    const char* post_gamma;
    const char* gamma;
    const float* post_rstd;
    const float* rstd;
    char* dR;
    char* dX;  // null: not wanted
    float* dgamma;
    char* dgate;  // channel: float[D]; row: float[N]; full: N x D in the rows' type
    float* dpost_gamma;
    int64_t lddy, lddh, ldh, ldx, ldg, lddr, lddx, lddg, N, D;
    int gate_kind;
    float scale;
};

constexpr int64_t kResNormMaxD = 32768;  // a row of the forward as floats in shared memory

// Groups of rows that the two gradients which are summed over the rows have partial sums of, at most: one a row, 16 MB
// each, and 16 an SM.  The backward has as many as are resident at once (rows over a cluster far fewer), or 128.
constexpr int kResNormColsGroups = 128, kResNormMaxGroups = 2432;
inline int resnorm_groups(int64_t N, int64_t D) {
    static_assert((1 << 22) / kResNormMaxD >= kResNormColsGroups, "the groups of the longest rows");
    const int64_t room = (1 << 22) / D, most = room < kResNormMaxGroups ? room : kResNormMaxGroups;
    return static_cast<int>(N < 1 ? 1 : N < most ? N : most);
}
// What a row's elements need of the row's sums, where those are taken first (residual_norm.cu).
struct RowStats {
    float k1, k2;
};
inline size_t resnorm_workspace_bytes(int64_t N, int64_t D) {
    const size_t part = static_cast<size_t>(resnorm_groups(N, D)) * static_cast<size_t>(D) * 4;
    return (2 * part + static_cast<size_t>(N) * sizeof(RowStats) + 255) / 256 * 256;
}

cudaError_t launch_resnorm_fwd(int es, const ResNormFwd& a, cudaStream_t s);
cudaError_t launch_resnorm_bwd(int es, const ResNormBwd& a, void* workspace, cudaStream_t s);

}  // namespace foak
