// block_norm.hip -- the norm behind a block with its gate and the scaled residual, and the norm in front of
// the next block, in one pass, and its backward pass (include/gdr.h: gdr_block_norm_fwd, _bwd).
//
// Per row x in R^d, with kappa = 1 (L2) or 1 / d (RMS):
//     r = (kappa sum x^2 + eps)^{-1/2},  u = r w (.) x,  a = act(z)
//     h = res_scale res + scale a (.) u,   y = h
//     r2 = (kappa2 sum h^2 + eps)^{-1/2},  n = r2 w2 (.) h
// Backward, everything formed again from the inputs:
//     t2 = w2 (.) dn,  dh = dy + r2 t2 - kappa2 r2^3 (t2 . h) h,  dw2 = sum r2 dn (.) h
//     dres = res_scale dh,  g = scale dh,  dz = g (.) u (.) act'(z)
//     t = w (.) a (.) g,  dx = r t - kappa r^3 (t . x) x,  dw = sum r a (.) g (.) x
#include "block_norm.hpp"

#include <algorithm>

#include "gdr_device.hpp"
#include "gdr_mfma.hpp"

namespace gdr {
namespace {

constexpr int kThreads = 256;
constexpr int kWide = 512;  // most threads of a row
constexpr int E = 8;  // channels of a lane's piece

typedef uint32_t wu4 __attribute__((ext_vector_type(4), aligned(2)));

// Eight elements as they are stored, from an element-aligned address.
template <bool BF>
struct Piece {
    uint32_t w[BF ? 4 : 8];
    __device__ __forceinline__ void load(const void *base, long at, bool there) {
        const char *p = static_cast<const char *>(base) + at * (BF ? 2 : 4);
#pragma unroll
        for (int k = 0; k < (BF ? 4 : 8); k += 4) {
            wu4 a = {0, 0, 0, 0};
            if (there) a = *reinterpret_cast<const wu4 *>(p + 4 * k);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[k + i] = a[i];
        }
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (BF) return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        return __uint_as_float(w[i]);
    }
};

template <bool BF>
__device__ __forceinline__ void put(void *base, long at, const float (&x)[E]) {
    char *p = static_cast<char *>(base) + at * (BF ? 2 : 4);
    if constexpr (BF) {
        *reinterpret_cast<wu4 *>(p) = (wu4){pk_bf16(x[0], x[1]), pk_bf16(x[2], x[3]), pk_bf16(x[4], x[5]), pk_bf16(x[6], x[7])};
    } else {
#pragma unroll
        for (int k = 0; k < 8; k += 4)
            *reinterpret_cast<wu4 *>(p + 4 * k) = (wu4){__float_as_uint(x[k]), __float_as_uint(x[k + 1]), __float_as_uint(x[k + 2]),
                                                        __float_as_uint(x[k + 3])};
    }
}

// act(z) and its slope, from m = e^{-|z|}: the sigmoid and its complement are 1 / (1 + m) and m / (1 + m), neither
// formed by subtracting the other.  e^x is 2^(x log2 e), by the hardware's 2^t, times 1 + (what rounding t left out) ln 2;
// the reciprocal is the hardware's with one Newton step.  (The library's e^x and division made the backward pass of
// 4 x 4,096 x 16 heads of 128 bound by arithmetic, 147 us.)
__device__ __forceinline__ void activation(int act, float z, float &a, float &slope) {
    if (act == 0) {
        a = z;
        slope = 1.f;
        return;
    }
    constexpr float log2e = 1.44269504f, ln2 = 0.69314718f;
    const float x = -fabsf(z), u = x * log2e;
    float m = __builtin_amdgcn_exp2f(u);
    if (u > -150.f) m = fmaf(m, fmaf(x, log2e, -u) * ln2, m);  // else 0, and the difference may be infinite
    const float d = 1.f + m, r0 = __builtin_amdgcn_rcpf(d), big = fmaf(fmaf(-d, r0, 1.f), r0, r0), small = m * big;
    const float s = z < 0.f ? small : big, c = z < 0.f ? big : small;
    if (act == 1) {
        a = s;
        slope = s * c;
    } else {
        const bool far = x == -INFINITY;  // z s and z c of an infinite z
        a = far ? fmaxf(z, 0.f) : z * s;
        slope = far ? s : s * fmaf(z, c, 1.f);
    }
}

__device__ __forceinline__ float inverse(float kappa, float ss, float eps) {
    const float m = fmaf(kappa, ss, eps);
    return m > 0.f || m != m ? 1.f / sqrtf(m) : 0.f;
}

constexpr int kWaves = kWide / 64;

// Sums of N values over a row's lanes: P of a wave (P a power of two), or the whole workgroup with WIDE, through
// `room`, of which successive sums use different thirds.
template <bool WIDE, int N>
__device__ __forceinline__ void row_sum(float (&x)[N], int P, float (*room)[2 * kWaves], int &third) {
#pragma unroll
    for (int i = 0; i < N; ++i)
        for (int s = 1; s < (WIDE ? 64 : P); s <<= 1) x[i] += __shfl_xor(x[i], s);
    if constexpr (WIDE) {
        const int waves = blockDim.x >> 6;
        if (waves > 1) {
            if ((threadIdx.x & 63) == 0)
#pragma unroll
                for (int i = 0; i < N; ++i) room[third][(threadIdx.x >> 6) * 2 + i] = x[i];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < N; ++i) {
                x[i] = 0.f;
                for (int w = 0; w < waves; ++w) x[i] += room[third][w * 2 + i];
            }
            third = third == 2 ? 0 : third + 1;
        }
    }
}

// A lane's pieces of one row, as stored.
template <bool BF, int NV, bool BWD>
struct Row {
    Piece<BF> x[NV], z[NV], r[NV], dy[BWD ? NV : 1], dn[BWD ? NV : 1];
    __device__ __forceinline__ void load(const NormParams &p, uint32_t row, bool live, int lane, int P) {
        const uint32_t token = row / (uint32_t)p.H, head = row - token * p.H;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int ch = (v * P + lane) * E;
            const bool there = live && ch < p.d;
            const long c = (long)head * p.d + ch;
            x[v].load(p.x, token * p.ldx + c, there);
            if (p.z) z[v].load(p.z, token * p.ldz + c, there);
            if (p.res) r[v].load(p.res, token * p.ldr + c, there);
            if constexpr (BWD) {
                dy[v].load(p.dy, (long)row * p.d + ch, there);
                if (p.next) dn[v].load(p.dn, (long)row * p.d + ch, there);
            }
        }
    }
};

// NV pieces per lane.  WIDE: a workgroup per row; else P lanes.  A workgroup stays for many rows, with the weights
// in registers, and asks for a row while it works on the one before.
// Whole rows are bound by HBM: 65,536 rows of 2,048 bf16 with a residual and both norms 221 us, 4.9 TB/s (a workgroup to a row,
// which read the weights each time, 537).  Heads with a gate are bound by arithmetic: 262,144 of 128 channels take 48 us forward (4.2
// TB/s), 41 of them for 48 vector instructions an element, and 98 backward (3.4 TB/s), 65 of them for 75.
template <bool BF, int NV, bool WIDE, bool BWD>
__global__ void __launch_bounds__(WIDE ? kWide : kThreads) block_norm_kernel(NormParams p) {
    __shared__ float room[3][2 * kWaves];
    const int P = WIDE ? blockDim.x : p.lanes, groups = WIDE ? 1 : kThreads / P;
    const int lane = WIDE ? threadIdx.x : threadIdx.x % P, gl = WIDE ? 0 : threadIdx.x / P;
    int third = 0;
    float w[NV][E], w2[NV][E], sw[BWD ? NV : 1][E], sw2[BWD ? NV : 1][E];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int ch = (v * P + lane) * E;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            w[v][e] = p.w && ch < p.d ? ld_elem(p.w, ch + e, p.w_bf16) : 1.f;
            w2[v][e] = p.w2 && ch < p.d ? ld_elem(p.w2, ch + e, p.w_bf16) : 1.f;
            if constexpr (BWD) sw[v][e] = sw2[v][e] = 0.f;
        }
    }
    const uint32_t rows = (uint32_t)p.rows, step = gridDim.x * groups;
    constexpr bool kAhead = !BWD || NV == 1;  // two pieces of every tensor twice are more than the registers
    Row<BF, NV, BWD> next;
    uint32_t row = blockIdx.x * groups + gl;
    if constexpr (kAhead) next.load(p, row, row < rows, lane, P);
    for (uint32_t first = blockIdx.x * groups; first < rows; first += step, row += step) {
        const bool live = row < rows;
        if constexpr (!kAhead) next.load(p, row, live, lane, P);
        const Row<BF, NV, BWD> in = next;
        if (kAhead && first + step < rows) next.load(p, row + step, row + step < rows, lane, P);
        float ss[1] = {0.f};
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < E; ++e) ss[0] = fmaf(in.x[v].get(e), in.x[v].get(e), ss[0]);
        float r = 1.f;
        if (p.norm) {
            row_sum<WIDE, 1>(ss, P, room, third);
            r = inverse(p.kappa, ss[0], p.eps);
        }
        float h[NV][E], a[NV][E], slope[NV][E], both[2] = {0.f, 0.f};
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                a[v][e] = 1.f;
                slope[v][e] = 0.f;
                if (p.z) activation(p.act, in.z[v].get(e), a[v][e], slope[v][e]);
                h[v][e] = p.scale * (a[v][e] * (in.x[v].get(e) * r * w[v][e]));
                if (p.res) h[v][e] = fmaf(p.res_scale, in.r[v].get(e), h[v][e]);
                both[0] = fmaf(h[v][e], h[v][e], both[0]);
                if constexpr (BWD) {
                    if (p.next) both[1] = fmaf(in.dn[v].get(e) * w2[v][e], h[v][e], both[1]);
                }
            }
        float r2 = 0.f;
        if (p.next) {
            row_sum<WIDE, 2>(both, P, room, third);
            r2 = inverse(p.next_kappa, both[0], p.eps);
        }
        if constexpr (!BWD) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int ch = (v * P + lane) * E;
                if (!live || ch >= p.d) continue;
                put<BF>(p.y, (long)row * p.d + ch, h[v]);
                if (!p.next) continue;
#pragma unroll
                for (int e = 0; e < E; ++e) h[v][e] = h[v][e] * r2 * w2[v][e];
                put<BF>(p.n, (long)row * p.d + ch, h[v]);
            }
        } else {
            // of r2 h; r2^2 would pass fp32's range in a row of zeros with an eps below 2^-128
            const float back = p.next_kappa * r2 * (r2 * both[1]);
            float dot[1] = {0.f};
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    float dh = in.dy[v].get(e);
                    if (p.next) {
                        const float dn = in.dn[v].get(e);
                        sw2[v][e] = fmaf(dn, r2 * h[v][e], sw2[v][e]);
                        dh += r2 * (dn * w2[v][e] - back * h[v][e]);
                    }
                    const float hat = in.x[v].get(e) * r, g = p.scale * dh, ga = g * a[v][e];
                    slope[v][e] *= g * (hat * w[v][e]);
                    h[v][e] = dh;
                    sw[v][e] = fmaf(ga, hat, sw[v][e]);
                    a[v][e] = ga * w[v][e];
                    dot[0] = fmaf(a[v][e], hat, dot[0]);
                }
            if (p.norm) row_sum<WIDE, 1>(dot, P, room, third);
            const float k = p.norm ? p.kappa * dot[0] * r : 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int ch = (v * P + lane) * E;
                if (!live || ch >= p.d) continue;
                const long o = (long)row * p.d + ch;
                if (p.res) {
#pragma unroll
                    for (int e = 0; e < E; ++e) h[v][e] *= p.res_scale;
                    put<BF>(p.dres, o, h[v]);
                }
                if (p.z) put<BF>(p.dz, o, slope[v]);
#pragma unroll
                for (int e = 0; e < E; ++e) a[v][e] = r * (a[v][e] - k * in.x[v].get(e));
                put<BF>(p.dx, o, a[v]);
            }
        }
    }
    if constexpr (BWD) {
        // the workgroup's sums of the weight gradients
        for (int m = 0; m < 2; ++m) {
            if (!(m ? p.dw2 : p.dw)) continue;  // uniform
            float *out = p.partial + ((long)m * gridDim.x + blockIdx.x) * p.d;
            if constexpr (WIDE) {
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const int ch = (v * P + lane) * E;
                    if (ch < p.d)
#pragma unroll
                        for (int e = 0; e < E; ++e) out[ch + e] = m ? sw2[v][e] : sw[v][e];
                }
            } else {
                __shared__ float sum[kThreads / 64][64 * E];
                __syncthreads();
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    float x = m ? sw2[0][e] : sw[0][e];
                    for (int s = P; s < 64; s <<= 1) x += __shfl_xor(x, s);
                    if ((threadIdx.x & 63) < P) sum[threadIdx.x >> 6][lane * E + e] = x;
                }
                __syncthreads();
                for (int ch = threadIdx.x; ch < p.d; ch += kThreads) {
                    float x = 0.f;
                    for (int k = 0; k < kThreads / 64; ++k) x += sum[k][ch];
                    out[ch] = x;
                }
            }
        }
    }
}

// The workgroups' sums, always in the same order: 16 channels per workgroup, 64 rows of threads.
__global__ void __launch_bounds__(256) block_norm_weight_kernel(NormParams p) {
    __shared__ f32x4 part[64][4];
    float *dw = blockIdx.y ? p.dw2 : p.dw;
    if (!dw) return;
    const float *from = p.partial + (long)blockIdx.y * p.blocks * p.d;
    const int cl = threadIdx.x & 3, rl = threadIdx.x >> 2, ch = blockIdx.x * 16 + cl * 4;
    f32x4 a = {0.f, 0.f, 0.f, 0.f};
    if (ch < p.d) {  // d is a multiple of 8
#pragma unroll 4
        for (int b = rl; b < p.blocks; b += 64) a += *reinterpret_cast<const f32x4 *>(from + (long)b * p.d + ch);
    }
    part[rl][cl] = a;
    for (int k = 32; k > 0; k >>= 1) {
        __syncthreads();
        if (rl < k) part[rl][cl] += part[rl + k][cl];
    }
    if (rl == 0 && ch < p.d) {
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[ch + i] = part[0][cl][i];
    }
}

template <bool BF, bool BWD>
const void *pick(int nv, bool wide) {
    if (!wide) return reinterpret_cast<const void *>(&block_norm_kernel<BF, 1, false, BWD>);
    return nv == 1   ? reinterpret_cast<const void *>(&block_norm_kernel<BF, 1, true, BWD>)
                     : reinterpret_cast<const void *>(&block_norm_kernel<BF, 2, true, BWD>);
}

// Workgroups at most, so that each stays for many rows of a large call.  They are more than the chip holds at once: of 256 threads
// with one piece a lane 5 fit a compute unit forward (88 registers; fp32 112: 4) and 3 backward (137; fp32 161), 1,280 and 768 on 256
// units, so some start when others have ended.  Forward that costs nothing (1,280: heads 48 us, join 222, as with 2,048);
// backward it does (768: heads of 128 81 us against 98, the fp32 join of 2,331 x 1,000 22 against 24).
constexpr int kBlocks = 2048, kBlocksBwd = 1024;

struct Plan {
    bool wide;
    int nv, threads;
};

Plan plan(NormParams &p, bool bwd) {
    Plan r;
    const int pieces = p.d / E;
    r.wide = pieces > 64;
    r.nv = pieces <= kWide ? 1 : 2;
    r.threads = r.wide ? ((pieces + r.nv - 1) / r.nv + 63) / 64 * 64 : kThreads;
    p.lanes = 1;
    while (!r.wide && p.lanes < pieces) p.lanes <<= 1;
    const int64_t groups = r.wide ? 1 : kThreads / p.lanes, blocks = (p.rows + groups - 1) / groups;
    const int most = (bwd ? kBlocksBwd : kBlocks) * kThreads / r.threads;
    p.blocks = (int)std::min<int64_t>(blocks, most);
    return r;
}

}  // namespace

size_t block_norm_workspace(const NormParams &p0) {
    NormParams p = p0;
    plan(p, true);
    return (size_t)p.blocks * p.d * 2 * sizeof(float);
}

hipError_t launch_block_norm(const NormParams &p0, bool bwd, hipStream_t s) {
    NormParams p = p0;
    const Plan r = plan(p, bwd);
    void *args[] = {&p};
    const void *fn = p.io_bf16 ? (bwd ? pick<true, true>(r.nv, r.wide) : pick<true, false>(r.nv, r.wide))
                               : (bwd ? pick<false, true>(r.nv, r.wide) : pick<false, false>(r.nv, r.wide));
    hipError_t e = p.blocks > 0 ? hipLaunchKernel(fn, dim3((unsigned)p.blocks), dim3((unsigned)r.threads), args, 0, s) : hipSuccess;
    if (e == hipSuccess && bwd && (p.dw || p.dw2))
        e = hipLaunchKernel(reinterpret_cast<const void *>(&block_norm_weight_kernel), dim3((unsigned)((p.d + 15) / 16), 2), dim3(256), args, 0, s);
    return e;
}

}  // namespace gdr
