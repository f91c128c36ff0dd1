// block_norm.hpp -- parameter block and launchers of the block norm (block_norm.hip), shared with its entry
// points (delta_api.hip).  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdr {

constexpr int kMaxNormWidth = 8192;  // channels of a row

// Parameters of one call; rows are (token, head), `ld*` elements between tokens.
struct NormParams {
    int64_t rows;
    int H, d;
    int io_bf16, w_bf16;
    int norm, next, act;  // gdr_norm, whether the following norm is formed, gdr_act
    float kappa, next_kappa, eps, scale, res_scale;
    const void *x, *z, *res, *w, *w2;  // all but x may be NULL
    int64_t ldx, ldz, ldr;
    void *y, *n;
    const void *dy, *dn;  // dense
    void *dx, *dz, *dres;
    float *dw, *dw2;      // [d] or NULL
    float *partial;       // sums of the workgroups, dw's and then dw2's
    int lanes, blocks;    // set by the launcher
};

size_t block_norm_workspace(const NormParams &p);
hipError_t launch_block_norm(const NormParams &p, bool bwd, hipStream_t s);

}  // namespace gdr
