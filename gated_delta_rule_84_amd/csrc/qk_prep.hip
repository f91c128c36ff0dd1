// qk_prep.hip -- norms of queries and keys per head with the position rotation in the same
// pass, and its backward pass (include/gdr.h: gdr_qk_prep_fwd, gdr_qk_prep_bwd).
//
// One row x in R^d per (token, head).  Forward, with kappa = 1 (L2) or 1/d (RMS):
//     r = (kappa sum x^2 + eps)^{-1/2}   (0 where the bracket is 0; 1 without a norm)
//     n = r w (.) x,   out = scale Rot_pos(n)
// Rot turns channel pair i < rot/2 by theta = pos f_i and multiplies it by rot_scale.
// Backward, from g = d loss / d out:
//     m = scale Rot_pos^T(g),  t = w (.) m,  dw = sum over rows r m (.) x
//     dx = r t - kappa r^3 (t . x) x
// and without a norm dx = m, which x does not enter: the forward pass of g, turned the other way.
//
// Bound by HBM (forward 2 and backward 3 passes over the heads, under 10 operations per
// byte), so the layout serves the loads.  Rotated channels are held as pairs: a lane owns
// VP = 4 consecutive pairs of a row, read from the two places where the pairs' members lie
// (8 bytes each of bf16, 16 of fp32; interleaved members in one access of twice that), so the
// rotation needs no exchange between lanes; P = 2^k lanes hold a row and only the norm's sum
// crosses lanes (log2 P xor shuffles).  A group of P lanes works on up to 8 heads of one
// token, each loaded while the one before it is worked on, and the workgroup forms the
// cosines and sines of its tokens once, in shared memory (each lane its own pairs' before:
// 5 us of 91 in the backward pass below).
// 4 x 4,096 tokens of 16 + 16 heads of 128, weights, full rotation, median kernel times: bf16 forward
// 47 us (5.7 TB/s), backward 87 us (4.6 TB/s) and 4.8 us for the weights' sums, 44 us in all without a
// norm; 65,536 tokens of 32 + 8 bf16 forward 254 us (5.3 TB/s); fp32 forward 111 us (4.8 TB/s), backward
// with its sums 163 us (4.9 TB/s).  8 tokens of 16 + 16 take 4.1 us, which is a launch and one trip to memory.
// Half rotations of rot_dim / 2 not a multiple of 4 take each member by itself, all lanes for the sake of
// the one at the end of the rotated part: 1.6 to 3.3 TB/s.  P is rounded up to a power of two, so heads
// whose d / 8 is none leave lanes idle: of 65,536 tokens of 16 + 4 heads, bf16 heads of 80, 96, 136 and 192 are
// done at 3.8, 4.4, 3.7 and 4.7 TB/s forward, at 3.5, 4.1, 3.0 and 4.0 backward; fp32 ones at 4.7 or more.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gdr_device.hpp"
#include "gdr_mfma.hpp"
#include "mixer.hpp"

namespace gdr {
namespace {

constexpr int kThreads = 256;
constexpr int VP = 4;  // pairs per lane

// N elements of a row as they are stored, from an element-aligned address (the hardware takes
// a global access of a dword or more at any byte address).
template <bool BF, int N>
struct Elems {
    static constexpr int W = BF ? N / 2 : N;
    uint32_t w[W];

    template <int K> struct Words { typedef uint32_t type __attribute__((ext_vector_type(K), aligned(2))); };
    static constexpr int K = W < 4 ? W : 4;  // words per access

    __device__ __forceinline__ void load(const void *base, long at) {
        const char *p = static_cast<const char *>(base) + at * (BF ? 2 : 4);
#pragma unroll
        for (int k = 0; k < W; k += K) {
            const typename Words<K>::type a = *reinterpret_cast<const typename Words<K>::type *>(p + 4 * k);
#pragma unroll
            for (int i = 0; i < K; ++i) w[k + i] = a[i];
        }
    }
    __device__ __forceinline__ void store(void *base, long at) const {
        char *p = static_cast<char *>(base) + at * (BF ? 2 : 4);
#pragma unroll
        for (int k = 0; k < W; k += K) {
            typename Words<K>::type a;
#pragma unroll
            for (int i = 0; i < K; ++i) a[i] = w[k + i];
            *reinterpret_cast<typename Words<K>::type *>(p + 4 * k) = a;
        }
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (BF) return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        return __uint_as_float(w[i]);
    }
    // elements i and i + 1 (i even)
    __device__ __forceinline__ void set2(int i, float a, float b) {
        if constexpr (BF) {
            w[i / 2] = pk_bf16(a, b);
        } else {
            w[i] = __float_as_uint(a);
            w[i + 1] = __float_as_uint(b);
        }
    }
};

// Where a lane's pairs lie in the row.
//   kAdjacent  members side by side (interleaved rotation, or none): 2 VP elements at 2 i
//   kSplit     VP elements at one place and VP at another (half rotation whose rot / 2 is
//              a multiple of VP; lanes past it hold channels that are not rotated)
//   kScattered each member at a place of its own (half rotation, any even rot)
enum Layout { kAdjacent = 0, kSplit = 1, kScattered = 2 };

// A lane's pairs of one row, as stored.
template <bool BF, int LAY>
struct Held {
    Elems<BF, LAY == kAdjacent ? 2 * VP : VP> a, b;  // kAdjacent uses only a
    float e[LAY == kScattered ? VP : 1], o[LAY == kScattered ? VP : 1];
};

template <bool BF, int LAY>
struct Row {
    int at[2];      // kAdjacent: [0]; kSplit: both
    int i0, half;   // kScattered
    __device__ __forceinline__ void place(int pair0, int half_) {
        i0 = pair0;
        half = half_;
        if (LAY == kSplit && pair0 < half_) {
            at[0] = pair0;
            at[1] = pair0 + half_;
        } else {
            at[0] = 2 * pair0;
            at[1] = 2 * pair0 + VP;
        }
    }
    // channel of pair j's first / second member
    __device__ __forceinline__ int channel(int j, int second) const {
        if constexpr (LAY == kAdjacent) return at[0] + 2 * j + second;
        if constexpr (LAY == kSplit) return at[second] + j;
        const int i = i0 + j;
        return i < half ? i + (second ? half : 0) : 2 * i + second;
    }
    __device__ __forceinline__ void load(const void *base, long row, Held<BF, LAY> &r) const {
        if constexpr (LAY == kScattered) {
#pragma unroll
            for (int j = 0; j < VP; ++j) {
                r.e[j] = ld_elem(base, row + channel(j, 0), BF);
                r.o[j] = ld_elem(base, row + channel(j, 1), BF);
            }
        } else {
            r.a.load(base, row + at[0]);
            if constexpr (LAY == kSplit) r.b.load(base, row + at[1]);
        }
    }
    __device__ __forceinline__ void unpack(const Held<BF, LAY> &r, float (&e)[VP], float (&o)[VP]) const {
#pragma unroll
        for (int j = 0; j < VP; ++j) {
            if constexpr (LAY == kAdjacent) {
                e[j] = r.a.get(2 * j);
                o[j] = r.a.get(2 * j + 1);
            } else if constexpr (LAY == kSplit) {
                e[j] = r.a.get(j);
                o[j] = r.b.get(j);
            } else {
                e[j] = r.e[j];
                o[j] = r.o[j];
            }
        }
    }
    __device__ __forceinline__ void store(void *base, long row, const float (&e)[VP], const float (&o)[VP]) const {
        if constexpr (LAY == kScattered) {
#pragma unroll
            for (int j = 0; j < VP; ++j) {
                st_elem(base, row + channel(j, 0), e[j], BF);
                st_elem(base, row + channel(j, 1), o[j], BF);
            }
        } else {
            Held<BF, LAY> r;
#pragma unroll
            for (int j = 0; j < VP; j += 2) {
                if constexpr (LAY == kAdjacent) {
                    r.a.set2(2 * j, e[j], o[j]);
                    r.a.set2(2 * j + 2, e[j + 1], o[j + 1]);
                } else {
                    r.a.set2(j, e[j], e[j + 1]);
                    r.b.set2(j, o[j], o[j + 1]);
                }
            }
            r.a.store(base, row + at[0]);
            if constexpr (LAY == kSplit) r.b.store(base, row + at[1]);
        }
    }
};

// The weights of a lane's pairs, stored as bf16 (WB) or fp32.
template <bool WB, int LAY>
__device__ __forceinline__ void weights(const void *w, int pair0, int half, float (&we)[VP], float (&wo)[VP]) {
    Row<WB, LAY> at;
    Held<WB, LAY> h;
    at.place(pair0, half);
    at.load(w, 0, h);
    at.unpack(h, we, wo);
}

// sum over the P lanes of a row (P a power of two)
__device__ __forceinline__ float row_sum(float x, int P) {
    for (int s = 1; s < P; s <<= 1) x += __shfl_xor(x, s);
    return x;
}

// Cosine and sine of pos * f_i, times rot_scale and rot_sin; pairs past the rotated part get 1 and 0.  The
// angle is formed and reduced to a fraction of a turn in 64 bits: at position 10^6 its 32-bit
// product would be off by 0.06.
__device__ __forceinline__ float2 angle(const QkParams &p, unsigned token, int i) {
    if (2 * i >= p.rot) return make_float2(1.f, 0.f);
    const int pos = p.pos ? p.pos[token] : (int)(token % (unsigned)p.T);
    double turn = (double)pos * p.inv_freq[i] * 0.15915494309189535;
    turn -= rint(turn);
    float sn, cs;
    sincospif(2.f * (float)turn, &sn, &cs);
    return make_float2(cs * p.rot_scale, sn * p.rot_sin);
}

// r of one row from its sum of squares (already over the P lanes)
__device__ __forceinline__ float inverse_norm(const QkParams &p, float ss) {
    if (p.norm == 0) return 1.f;
    const float m = fmaf(p.kappa, ss, p.eps);
    return m > 0.f || m != m ? 1.f / sqrtf(m) : 0.f;
}

template <bool BF, int LAY, bool BWD>
__global__ void __launch_bounds__(kThreads) qk_prep_kernel(QkParams p) {
    __shared__ float2 turns[kThreads * VP];
    const bool isk = blockIdx.x >= (unsigned)p.blocks_q;
    const QkTensor &X = isk ? p.k : p.q;
    const long block = isk ? (long)blockIdx.x - p.blocks_q : blockIdx.x;
    const long nblocks = isk ? p.blocks_k : p.blocks_q;
    const int P = p.lanes, groups = kThreads / P;
    const int gl = threadIdx.x / P, lane = threadIdx.x % P;
    const int i0 = lane * VP;
    const bool holds = i0 < p.d / 2;  // lanes past the row only take part in the sums
    Row<BF, LAY> at;
    at.place(holds ? i0 : 0, p.rot / 2);
    float we[VP], wo[VP], ae[VP], ao[VP];
#pragma unroll
    for (int j = 0; j < VP; ++j) {
        we[j] = wo[j] = 1.f;
        ae[j] = ao[j] = 0.f;
    }
    if (X.w && p.w_bf16) weights<true, LAY>(X.w, holds ? i0 : 0, p.rot / 2, we, wo);
    else if (X.w) weights<false, LAY>(X.w, holds ? i0 : 0, p.rot / 2, we, wo);
    const int pairs = P * VP, shift = __ffs(pairs) - 1;
    const long items = p.tokens * X.slices;
    for (long first = block * groups; first < items; first += nblocks * groups) {
        // the workgroup's items are slices of a few tokens that follow each other
        const unsigned token0 = items >> 32 ? (unsigned)(first / X.slices) : (unsigned)first / (unsigned)X.slices;
        const unsigned at0 = (unsigned)(first - (long)token0 * X.slices), mine = at0 + gl, step = mine / X.slices;
        const int here = (int)min((long)groups, items - first);
        const long token = token0 + step;
        const int h0 = gl < here ? (int)(mine - step * X.slices) * p.rows : X.H, h1 = min(h0 + p.rows, X.H);
        // each row is loaded while the one before it is worked on, the first under the angles
        Held<BF, LAY> next, gnext;
        auto fetch = [&](int h) __attribute__((always_inline)) {
            at.load(X.x, token * X.ld + (long)h * p.d, next);
            if constexpr (BWD) at.load(X.g, (token * X.H + h) * p.d, gnext);
        };
        if (h0 < h1) fetch(h0);
        const int used = ((at0 + here - 1) / X.slices + 1) << shift;  // angles of these tokens, at most kThreads * VP
        float c[VP], s[VP];
        if (p.rot > 0) {
            for (int i = threadIdx.x; i < used; i += kThreads) turns[i] = angle(p, token0 + (i >> shift), i & (pairs - 1));
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < VP; ++j) {
            const float2 t = p.rot > 0 ? turns[gl < here ? ((int)step << shift) + i0 + j : 0] : make_float2(1.f, 0.f);
            c[j] = t.x;
            s[j] = t.y;
        }
        if (first + nblocks * groups < items) __syncthreads();  // before the next angles
        for (int h = h0; h < h1; ++h) {
            const long out = (token * X.H + h) * p.d;
            float e[VP], o[VP], ge[VP], go[VP];
            at.unpack(next, e, o);
            if constexpr (BWD) at.unpack(gnext, ge, go);
            if (h + 1 < h1) fetch(h + 1);
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < VP; ++j) ss = fmaf(e[j], e[j], fmaf(o[j], o[j], ss));
            if (!holds) ss = 0.f;
            const float r = inverse_norm(p, row_sum(ss, P));
            if constexpr (!BWD) {
                const float rs = r * X.scale;
#pragma unroll
                for (int j = 0; j < VP; ++j) {
                    const float ne = e[j] * rs * we[j], no = o[j] * rs * wo[j];
                    e[j] = c[j] * ne - s[j] * no;
                    o[j] = s[j] * ne + c[j] * no;
                }
            } else {
                float dot = 0.f;
#pragma unroll
                for (int j = 0; j < VP; ++j) {
                    const float me = X.scale * (c[j] * ge[j] + s[j] * go[j]);
                    const float mo = X.scale * (c[j] * go[j] - s[j] * ge[j]);
                    const float xe = r * e[j], xo = r * o[j];
                    ae[j] = fmaf(me, xe, ae[j]);
                    ao[j] = fmaf(mo, xo, ao[j]);
                    ge[j] = me * we[j];
                    go[j] = mo * wo[j];
                    dot = fmaf(ge[j], xe, fmaf(go[j], xo, dot));
                    e[j] = xe;
                    o[j] = xo;
                }
                if (!holds) dot = 0.f;
                dot = p.kappa * row_sum(dot, P);
#pragma unroll
                for (int j = 0; j < VP; ++j) {
                    e[j] = r * fmaf(-dot, e[j], ge[j]);
                    o[j] = r * fmaf(-dot, o[j], go[j]);
                }
            }
            if (holds) at.store(X.out, out, e, o);
        }
    }
    if constexpr (BWD) {
        if (!X.dw) return;  // uniform over the workgroup
        __shared__ float sum[kThreads / 64][256];
        const int wave = threadIdx.x >> 6;
#pragma unroll
        for (int j = 0; j < VP; ++j) {
            for (int k = P; k < 64; k <<= 1) {
                ae[j] += __shfl_xor(ae[j], k);
                ao[j] += __shfl_xor(ao[j], k);
            }
            if (holds && (threadIdx.x & 63) < P) {
                sum[wave][at.channel(j, 0)] = ae[j];
                sum[wave][at.channel(j, 1)] = ao[j];
            }
        }
        __syncthreads();
        for (int ch = threadIdx.x; ch < p.d; ch += kThreads) {
            float a = 0.f;
            for (int w = 0; w < kThreads / 64; ++w) a += sum[w][ch];
            p.partial[(long)blockIdx.x * p.d + ch] = a;
        }
    }
}

// The workgroups' sums of the weight gradients, always in the same order: 16 channels per
// block, 4 lanes of 4 channels in 64 rows of threads.  4.6 us for 2 x 768 sums of 128 channels
// (0.8 MB, in cache: a launch and 12 dependent rows of loads per thread).
__global__ void __launch_bounds__(256) qk_weight_kernel(QkParams p) {
    __shared__ f32x4 part[64][4];
    const bool isk = blockIdx.y != 0;
    float *dw = isk ? p.k.dw : p.q.dw;
    if (!dw) return;
    const int cl = threadIdx.x & 3, rl = threadIdx.x >> 2, ch = blockIdx.x * 16 + cl * 4;
    const int first = isk ? p.blocks_q : 0, n = isk ? p.blocks_k : p.blocks_q;
    f32x4 a = {0.f, 0.f, 0.f, 0.f};
    if (ch < p.d) {  // d is a multiple of 8
#pragma unroll 4
        for (int b = rl; b < n; b += 64) a += *reinterpret_cast<const f32x4 *>(p.partial + (long)(first + b) * p.d + ch);
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
const void *pick_layout(int lay) {
    switch (lay) {
    case kAdjacent: return reinterpret_cast<const void *>(&qk_prep_kernel<BF, kAdjacent, BWD>);
    case kSplit: return reinterpret_cast<const void *>(&qk_prep_kernel<BF, kSplit, BWD>);
    default: return reinterpret_cast<const void *>(&qk_prep_kernel<BF, kScattered, BWD>);
    }
}

constexpr int kMaxBlocks = 768;  // workgroups per tensor of a backward pass: about what the chip holds at once
constexpr int kMaxGrid = (1 << 23) - 1;  // of a forward pass: a launch of both tensors has fewer than 2^32 threads

// Lanes, heads per group and workgroups of one call; returns its layout.
int plan(QkParams &p, bool bwd) {
    const int half = p.rot / 2;
    const int lay = !p.half_layout || half == 0 ? kAdjacent : (half % VP == 0 ? kSplit : kScattered);
    p.lanes = 1;
    while (p.lanes * VP < p.d / 2) p.lanes <<= 1;
    const int groups = kThreads / p.lanes;
    // Up to 8 heads share a token's angles and follow each other in the pipeline of loads; fewer
    // where that leaves the chip's 1024 SIMDs without 4 waves each and latency is what counts.
    const long rows = p.tokens * (p.q.H > p.k.H ? p.q.H : p.k.H) * p.lanes / 64;
    p.rows = 8;
    while (p.rows > 1 && rows / p.rows < 4096) p.rows >>= 1;
    QkTensor *all[] = {&p.q, &p.k};
    long blocks[2];
    for (int i = 0; i < 2; ++i) {
        all[i]->slices = (all[i]->H + p.rows - 1) / p.rows;
        blocks[i] = (p.tokens * all[i]->slices + groups - 1) / groups;
        blocks[i] = std::min<long>(blocks[i], bwd ? kMaxBlocks : kMaxGrid);
    }
    p.blocks_q = (int)blocks[0];
    p.blocks_k = (int)blocks[1];
    return lay;
}

}  // namespace

size_t qk_prep_bwd_workspace(const QkParams &p0) {
    QkParams p = p0;
    plan(p, true);
    return (size_t)(p.blocks_q + p.blocks_k) * p.d * sizeof(float);
}

hipError_t launch_qk_prep(const QkParams &p0, bool bwd, hipStream_t s) {
    QkParams p = p0;
    p.rot_sin = p.rot_scale;
    if (bwd && p.norm == 0) {
        // without a norm dx = scale Rot^T(g): the gradient's forward pass with its turns the other way, and x is not read
        for (QkTensor *X : {&p.q, &p.k}) {
            X->x = X->g;
            X->ld = (int64_t)X->H * p.d;
        }
        p.rot_sin = -p.rot_scale;
        bwd = false;
    }
    const int lay = plan(p, bwd);
    const long blocks = (long)p.blocks_q + p.blocks_k;
    void *args[] = {&p};
    const void *fn = p.io_bf16 ? (bwd ? pick_layout<true, true>(lay) : pick_layout<true, false>(lay))
                               : (bwd ? pick_layout<false, true>(lay) : pick_layout<false, false>(lay));
    hipError_t e = blocks > 0 ? hipLaunchKernel(fn, dim3((unsigned)blocks), dim3(kThreads), args, 0, s) : hipSuccess;
    if (e == hipSuccess && bwd && (p.q.dw || p.k.dw))
        e = hipLaunchKernel(reinterpret_cast<const void *>(&qk_weight_kernel), dim3((unsigned)((p.d + 15) / 16), 2),
                            dim3(256), args, 0, s);
    return e;
}

}  // namespace gdr
