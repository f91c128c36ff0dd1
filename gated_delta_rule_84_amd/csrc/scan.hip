// scan.hip -- gated linear recurrence: the single-token step (see scan_impl.hpp).
#include "scan_impl.hpp"

namespace gdr {
namespace {

// Words at an element-aligned address (the hardware takes a global access of a dword or more at
// any byte address); n of the V elements, one by one where that is not all of them.
typedef uint32_t w2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t w4 __attribute__((ext_vector_type(4), aligned(2)));

template <bool BF>
__device__ __forceinline__ void load_at(Pack<BF> &x, const void *base, int64_t at, int n) {
    constexpr int N = Pack<BF>::N;
    const char *p = static_cast<const char *>(base) + at * x.es;
    if (n < V) {
#pragma unroll
        for (int k = 0; k < N; ++k) x.w[k] = 0;
        for (int v = 0; v < n; ++v) {
            const uint32_t e = BF ? reinterpret_cast<const uint16_t *>(p)[v] : reinterpret_cast<const uint32_t *>(p)[v];
#pragma unroll
            for (int k = 0; k < N; ++k) x.w[k] |= k == (BF ? v / 2 : v) ? (BF && (v & 1) ? e << 16 : e) : 0;
        }
    } else if constexpr (N == 2) {
        const w2 a = *reinterpret_cast<const w2 *>(p);
        x.w[0] = a[0];
        x.w[1] = a[1];
    } else {
#pragma unroll
        for (int k = 0; k < N; k += 4) {
            const w4 a = *reinterpret_cast<const w4 *>(p + 4 * k);
#pragma unroll
            for (int i = 0; i < 4; ++i) x.w[k + i] = a[i];
        }
    }
}

template <bool BF>
__device__ __forceinline__ void store_at(const Pack<BF> &x, void *base, int64_t at, int n) {
    constexpr int N = Pack<BF>::N;
    char *p = static_cast<char *>(base) + at * x.es;
    if (n < V) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (v >= n) continue;
            if constexpr (BF) reinterpret_cast<uint16_t *>(p)[v] = (uint16_t)(x.w[v / 2] >> (16 * (v & 1)));
            else reinterpret_cast<uint32_t *>(p)[v] = x.w[v];
        }
    } else if constexpr (N == 2) {
        *reinterpret_cast<w2 *>(p) = (w2){x.w[0], x.w[1]};
    } else {
#pragma unroll
        for (int k = 0; k < N; k += 4) *reinterpret_cast<w4 *>(p + 4 * k) = (w4){x.w[k], x.w[k + 1], x.w[k + 2], x.w[k + 3]};
    }
}

// One token for every batch row: the state is read and written in place.  512 rows of 2,048 bf16
// channels with fp32 gates: 4.0 us for 16.8 MB, most of it in cache (4.2 TB/s; a launch alone takes
// over 2 us).  Each lane has 4 channels of one row, so short calls still spread over the chip.
template <bool IOB, bool GB, int F, bool LOG>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanParams p) {
    const unsigned groups = (p.D + V - 1) / V;
    const long i = (long)blockIdx.x * 256 + threadIdx.x, b = i / groups;
    const int ch = (int)(i - b * groups) * V, n = min(V, p.D - ch);
    if (b >= p.B) return;
    Pack<IOB> x;
    Pack<GB> al, be;
    Pack<false> S;
    float a[V], u[V], h[V];
    load_at(x, p.x, b * p.ldx + ch, n);
    load_at(al, p.alpha, b * p.lda + ch, n);
    if (F == kGiven) load_at(be, p.beta, b * p.ldb + ch, n);
    load_at(S, p.ST, b * p.D + ch, n);
    gates<F, LOG, GB>(al, be, a, u);
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = fmaf(a[v], S.get(v), u[v] * x.get(v));
#pragma unroll
    for (int v = 0; v < V; v += 2) {
        S.set2(v, h[v], h[v + 1]);
        x.set2(v, h[v], h[v + 1]);
    }
    store_at(S, p.ST, b * p.D + ch, n);
    store_at(x, p.y, b * p.D + ch, n);
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

// of either direction: the smallest groups need most
size_t scan_workspace(const ScanParams &p) { return (size_t)chain_bytes(p, kGroupPacked); }

long scan_threads(const ScanParams &p) { return columns_of(p) * p.nblk * 64 * waves_of(p); }

hipError_t launch_scan_copy(const float *src, float *dst, long n, hipStream_t s) {
    if (!dst || n == 0 || src == dst) return hipSuccess;
    void *args[] = {&src, &dst, &n};
    return hipLaunchKernel(reinterpret_cast<const void *>(&scan_copy_kernel), dim3((unsigned)((n + 255) / 256)), dim3(256),
                           args, 0, s);
}

hipError_t launch_scan_step(const ScanParams &p, hipStream_t s) {
    const long threads = (long)p.B * ((p.D + V - 1) / V);
    if ((threads + 255) / 256 > 0x7fffffffL) return hipErrorInvalidValue;
    ScanParams q = p;
    void *args[] = {&q};
    return hipLaunchKernel(pick<Step>(p), dim3((unsigned)((threads + 255) / 256)), dim3(256), args, 0, s);
}

}  // namespace gdr
