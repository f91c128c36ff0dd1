// delta_step.hip -- one token of the delta rule on resident states (delta.hpp).
//
// Per value head, with a = e^g:  d = beta (v - a S^T k),  o = a S^T q + d (k.q),  S' = a S + k d^T.
// Bound by HBM: a state is read and written once (8 bytes per element), everything else is small.  A
// thread holds 4 columns of R rows in registers between the sums over rows and the write-back.  512 requests of 16 heads of
// 128 x 128: 198 us, 5.5 TB/s; 8 requests of 32 heads, whose states stay in cache, 9.1 us.
#include "delta.hpp"

namespace gdr {
namespace {

typedef float nf4 __attribute__((ext_vector_type(4), aligned(4)));

// R rows per thread.  groups = dv / 4 column groups, rows_at = 256 / groups of them side by side.
template <int R>
__global__ void __launch_bounds__(256) delta_step_kernel(DeltaStepParams p, int groups, int rows_at) {
    __shared__ float sk[128], sq[128];
    __shared__ float red[8][256];
    const int hv = blockIdx.x % p.Hv, hk = hv / p.group, tid = threadIdx.x;
    const long b = blockIdx.x / p.Hv;
    const int cg = tid % groups, rt = tid / groups;
    const bool act = rt < rows_at;
    float *S = p.S + ((long)blockIdx.x * p.dk) * p.dv + 4 * cg;
    nf4 s[R];
#pragma unroll
    for (int m = 0; m < R; ++m) {
        const int row = rt + m * rows_at;
        s[m] = (nf4){0.f, 0.f, 0.f, 0.f};
        if (act && row < p.dk) s[m] = *reinterpret_cast<const nf4 *>(S + (long)row * p.dv);
    }
    for (int i = tid; i < p.dk; i += 256) {
        sk[i] = ld_elem(p.k, b * p.ldk + (long)hk * p.dk + i, p.io_bf16);
        sq[i] = ld_elem(p.q, b * p.ldq + (long)hk * p.dk + i, p.io_bf16);
    }
    const float a = expf(ld_elem(p.g, b * p.ldg + hv, p.gate_bf16)), beta = ld_elem(p.b, b * p.ldb + hv, p.gate_bf16);
    __syncthreads();
    float u[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, kq = 0.f;
#pragma unroll
    for (int m = 0; m < R; ++m) {
        const int row = min(rt + m * rows_at, p.dk - 1);  // rows past the end are zeros
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            u[c] = fmaf(s[m][c], sk[row], u[c]);
            u[4 + c] = fmaf(s[m][c], sq[row], u[4 + c]);
        }
    }
    for (int i = 0; i < p.dk; ++i) kq = fmaf(sk[i], sq[i], kq);
#pragma unroll
    for (int c = 0; c < 8; ++c) red[c][tid] = act ? u[c] : 0.f;
    __syncthreads();
    // each column group's sums over its row threads
#pragma unroll
    for (int c = 0; c < 8; ++c) u[c] = 0.f;
    for (int i = 0; i < rows_at; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) u[c] += red[c][i * groups + cg];
    if (!act) return;
    float d[4];
    const long vrow = b * p.ldv + (long)hv * p.dv + 4 * cg;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        d[c] = beta * (ld_elem(p.v, vrow + c, p.io_bf16) - a * u[c]);
        if (rt == 0) st_elem(p.o, (long)blockIdx.x * p.dv + 4 * cg + c, fmaf(d[c], kq, a * u[4 + c]), p.io_bf16);
    }
#pragma unroll
    for (int m = 0; m < R; ++m) {
        const int row = rt + m * rows_at;
        if (row >= p.dk) continue;
        const float k = sk[row];
        nf4 x;
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = fmaf(k, d[c], a * s[m][c]);
        *reinterpret_cast<nf4 *>(S + (long)row * p.dv) = x;
    }
}

}  // namespace

hipError_t launch_delta_step(const DeltaStepParams &p0, hipStream_t s) {
    DeltaStepParams p = p0;
    int groups = p.dv / 4, rows_at = 256 / groups;
    if (rows_at > p.dk) rows_at = p.dk;
    const int R = (p.dk + rows_at - 1) / rows_at;
    void *args[] = {&p, &groups, &rows_at};
    const void *fn = R <= 1   ? reinterpret_cast<const void *>(&delta_step_kernel<1>)
                     : R <= 4 ? reinterpret_cast<const void *>(&delta_step_kernel<4>)
                     : R <= 8 ? reinterpret_cast<const void *>(&delta_step_kernel<8>)
                              : reinterpret_cast<const void *>(&delta_step_kernel<16>);
    return hipLaunchKernel(fn, dim3((unsigned)p.B * p.Hv), dim3(256), args, 0, s);
}

}  // namespace gdr
