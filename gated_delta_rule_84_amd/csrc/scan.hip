// scan.hip -- gated linear recurrence: the single-token step (see scan_impl.hpp).
#include "scan_impl.hpp"

namespace gdr {
namespace {

// One token for every batch row: the state is read and written in place.
template <bool IOB, bool GB, int F, bool LOG>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanParams p) {
    constexpr int V = Shape<IOB, GB>::V;
    const unsigned groups = (p.D + V - 1) / V;
    const long i = (long)blockIdx.x * 256 + threadIdx.x, b = i / groups;
    const int ch = (int)(i - b * groups) * V, n = min(V, p.D - ch);
    if (b >= p.B) return;
    Pack<IOB, V> x;
    Pack<GB, V> al, be;
    float *S = p.ST + b * p.D + ch;
    float a[V], u[V], h[V];
    const char *px = static_cast<const char *>(p.x) + (b * p.ldx + ch) * (IOB ? 2 : 4);
    const char *pa = static_cast<const char *>(p.alpha) + (b * p.lda + ch) * (GB ? 2 : 4);
    const char *pb = static_cast<const char *>(p.beta) + (b * p.ldb + ch) * (GB ? 2 : 4);
    char *py = static_cast<char *>(p.y) + (b * p.D + ch) * (IOB ? 2 : 4);
    const bool whole = n == V;
    if (whole) {
        x.load(px);
        al.load(pa);
        if (F == kGiven) be.load(pb);
    } else {
        x.load(px, n);
        al.load(pa, n);
        if (F == kGiven) be.load(pb, n);
    }
    load_state<V>(S, n, h);
    gates<F, LOG, GB, V>(al, be, a, u);
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = fmaf(a[v], h[v], u[v] * x.get(v));
#pragma unroll
    for (int v = 0; v < V; v += 2) x.set2(v, h[v], h[v + 1]);
    store_state<V>(S, n, h);
    if (whole) x.store(py);
    else x.store(py, n);
}

// ST = S0 (or 0) of a call without tokens
__global__ void __launch_bounds__(256) scan_copy_kernel(const float *src, float *dst, long n) {
    const long i = (long)blockIdx.x * 256 + threadIdx.x;
    if (i < n) dst[i] = src ? src[i] : 0.f;
}

struct Step {
    template <bool IOB, bool GB, int F, bool LOG, bool>
    static const void *get() { return reinterpret_cast<const void *>(&scan_step_kernel<IOB, GB, F, LOG>); }
};

}  // namespace

size_t scan_workspace(const ScanParams &p) { return (size_t)chain_bytes(p); }

hipError_t launch_scan_copy(const float *src, float *dst, long n, hipStream_t s) {
    if (!dst || n == 0 || src == dst) return hipSuccess;
    void *args[] = {&src, &dst, &n};
    return hipLaunchKernel(reinterpret_cast<const void *>(&scan_copy_kernel), dim3((unsigned)((n + 255) / 256)), dim3(256),
                           args, 0, s);
}

hipError_t launch_scan_step(const ScanParams &p, hipStream_t s) {
    const Pick k = pick<Step>(p);
    const long threads = (long)p.B * ((p.D + k.V - 1) / k.V);
    if ((threads + 255) / 256 > 0x7fffffffL) return hipErrorInvalidValue;
    ScanParams q = p;
    void *args[] = {&q};
    return hipLaunchKernel(k.fn, dim3((unsigned)((threads + 255) / 256)), dim3(256), args, 0, s);
}

}  // namespace gdr
