// mixer.hpp -- parameter blocks and launcher declarations of the query / key preparation and of the
// gated linear recurrence, shared by their entry points (mixer_api.hip) and kernels.  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdr {

// One of the two tensors of heads of a query / key preparation call.
struct QkTensor {
    const void *x;  // [tokens, H, d], `ld` elements between tokens
    const void *w;  // [d] or NULL
    const void *g;  // backward: the gradient of the output, dense
    void *out;      // dense: the output, or the gradient of x
    float *dw;      // backward: [d] or NULL
    int64_t ld;
    int H;
    float scale;
    int slices;     // groups of heads per token (set by the launcher)
};

// Parameters of one query / key preparation call.
struct QkParams {
    int64_t tokens;
    int T, d, rot;
    int io_bf16, w_bf16;
    int norm;         // 0 none, 1 L2, 2 RMS
    int half_layout;  // pairs (i, i + rot / 2) instead of (2 i, 2 i + 1)
    float kappa, eps, rot_scale;
    float rot_sin;  // rot_scale, or its negative for turns the other way (set by the launcher)
    const int32_t *pos;  // [tokens] or NULL (the row's index in its sequence)
    const double *inv_freq;
    QkTensor q, k;
    float *partial;  // backward: the workgroups' sums of the weight gradients
    int lanes, rows, blocks_q, blocks_k;  // set by the launcher
};

// Most elements between tokens of a gated linear recurrence (and channels of one), so that a block
// of 256 tokens spans at most 2^30 bytes, and most bytes of the states of packed sequences.
constexpr int64_t kMaxRow = 1 << 20, kMaxStates = 1 << 30;

constexpr int64_t kMaxThreads = 0xffffffff;  // of one launch (workgroups times their threads)

// Parameters of one gated linear recurrence call (forward, backward or single step).
struct ScanParams {
    int B, T, D;  // D channels per token
    int io_bf16, gate_bf16;
    int log_gate, coupled;
    const void *x, *alpha, *beta;  // beta may be NULL
    int64_t ldx, lda, ldb;         // elements between tokens
    const int32_t *off;            // [nseq + 1] or NULL: borders of packed sequences
    int nseq;
    const float *S0;  // may be NULL
    void *y;
    float *ST;    // may be NULL
    float *ckpt;  // forward output (may be NULL), backward input
    const void *dy;
    const float *dST;  // may be NULL
    void *dx, *dalpha, *dbeta;
    float *dS0;  // may be NULL
    int nblk;    // blocks of tokens per sequence
    void *ws;
};

// Launchers (defined next to their kernels).  They only enqueue work.
size_t qk_prep_bwd_workspace(const QkParams &p);
hipError_t launch_qk_prep(const QkParams &p, bool bwd, hipStream_t s);
size_t scan_workspace(const ScanParams &p);
long scan_threads(const ScanParams &p);  // of a pass's launch
hipError_t launch_scan_fwd(const ScanParams &p, hipStream_t s);
hipError_t launch_scan_bwd(const ScanParams &p, hipStream_t s);
hipError_t launch_scan_copy(const float *src, float *dst, long n, hipStream_t s);  // src NULL: zeros
hipError_t launch_scan_step(const ScanParams &p, hipStream_t s);

}  // namespace gdr
