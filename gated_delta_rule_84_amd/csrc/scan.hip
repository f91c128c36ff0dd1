// scan.hip -- gated linear recurrence per channel: forward over long sequences, backward and
// the single-token step (include/gdr.h: gdr_scan_fwd, gdr_scan_bwd, gdr_scan_step).
//
//     h_t = a_t h_{t-1} + b_t x_t,   y_t = h_t        (per channel, state in fp32)
//
// A token is the affine map h -> a h + u with u = b x; maps compose associatively,
// (A2, U2) o (A1, U1) = (A2 A1, A2 U1 + U2), so a block of tokens is reduced in parallel.
// The backward pass is the same recurrence run from the end.  With G_t the gradient that
// token t hands to t - 1,
//     g_t = dy_t + G_{t+1},  G_t = a_t g_t        (G_{T+1} = dS_T, dS_0 = G_1)
//     dx = b g,  dbeta = g x,  da = g h_{t-1}  (- g x where b = 1 - a)
// and h_{t-1} is formed again inside each block from the state that the forward pass kept
// at the block's border, so no state of a token is stored or read.
//
// Layout: a workgroup takes blocks of 512 tokens x CH channels.  8 lanes hold a row of the
// block (V channels each: 16-byte loads, 128-byte rows of bf16) and a lane holds 8 tokens
// one after the other (a strand), all of its inputs in registers between the reduction and
// the second pass, so every input is read once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdr.h"
#include "gdr_device.hpp"
#include "gdr_internal.hpp"
#include "gdr_mfma.hpp"

namespace gdr {
namespace {

constexpr int kBlk = GDR_SCAN_BLOCK;  // tokens per block
constexpr int kL = 8;                 // tokens per strand
constexpr int kLR = 8;                // lanes per row
constexpr int kStrands = kBlk / kL;   // 64
constexpr int kThreads = kStrands * kLR;
constexpr int kWaves = kThreads / 64;

typedef uint32_t w2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t w4 __attribute__((ext_vector_type(4), aligned(2)));

// V elements of one token, packed as they are stored.
template <bool BF, int V>
struct Pack {
    static constexpr int N = BF ? V / 2 : V;
    uint32_t w[N];

    __device__ __forceinline__ float get(int v) const {
        if constexpr (BF) return (v & 1) ? __uint_as_float(w[v / 2] & 0xffff0000u) : __uint_as_float(w[v / 2] << 16);
        return __uint_as_float(w[v]);
    }
    // members v and v + 1 (v even)
    __device__ __forceinline__ void set2(int v, float a, float b) {
        if constexpr (BF) {
            w[v / 2] = pk_bf16(a, b);
        } else {
            w[v] = __float_as_uint(a);
            w[v + 1] = __float_as_uint(b);
        }
    }
    // `n` of the V elements are inside the row
    __device__ __forceinline__ void load(const void *base, int64_t at, int n) {
        if (n == V) {
            const char *p = static_cast<const char *>(base) + at * (BF ? 2 : 4);
            if constexpr (N == 2) {
                const w2 a = *reinterpret_cast<const w2 *>(p);
                w[0] = a[0];
                w[1] = a[1];
            } else {
#pragma unroll
                for (int k = 0; k < N; k += 4) {
                    const w4 a = *reinterpret_cast<const w4 *>(p + 4 * k);
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[k + i] = a[i];
                }
            }
        } else {
            clear();
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (v >= n) continue;
                if constexpr (BF)
                    w[v / 2] |= (uint32_t) static_cast<const uint16_t *>(base)[at + v] << (16 * (v & 1));
                else
                    w[v] = static_cast<const uint32_t *>(base)[at + v];
            }
        }
    }
    __device__ __forceinline__ void store(void *base, int64_t at, int n) const {
        if (n == V) {
            char *p = static_cast<char *>(base) + at * (BF ? 2 : 4);
            if constexpr (N == 2) {
                w2 a;
                a[0] = w[0];
                a[1] = w[1];
                *reinterpret_cast<w2 *>(p) = a;
            } else {
#pragma unroll
                for (int k = 0; k < N; k += 4) {
                    w4 a;
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[i] = w[k + i];
                    *reinterpret_cast<w4 *>(p + 4 * k) = a;
                }
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (v >= n) continue;
                if constexpr (BF)
                    static_cast<uint16_t *>(base)[at + v] = (uint16_t)(w[v / 2] >> (16 * (v & 1)));
                else
                    static_cast<uint32_t *>(base)[at + v] = w[v];
            }
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < N; ++k) w[k] = 0;
    }
};

// n of V floats
template <int V>
__device__ __forceinline__ void load_state(const float *p, int n, float (&f)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = p && v < n ? p[v] : 0.f;
}
template <int V>
__device__ __forceinline__ void store_state(float *p, int n, const float (&f)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (v < n) p[v] = f[v];
}

// Decay and input factor of one token and channel from the stored gate values.
template <bool BETA>
__device__ __forceinline__ void gates(const ScanParams &p, float raw, float beta, float &a, float &b) {
    a = p.log_gate ? expf(raw) : raw;
    b = BETA ? beta : (p.coupled ? (p.log_gate ? -expm1f(raw) : 1.f - raw) : 1.f);
}

// The tokens t0 .. t0 + 7 of a strand: bit j of `in` where the token belongs to a sequence,
// of `first` / `last` where it opens / closes one; seq[j] its sequence.  Offsets are read
// with sequence numbers clamped to 0 .. nseq, whatever they hold.
template <bool PACKED>
struct Marks {
    unsigned in = 0, first = 0, last = 0;
    int seq[PACKED ? kL : 1];

    __device__ __forceinline__ void find(const ScanParams &p, int b, long t0) {
        if constexpr (PACKED) {
            int lo = 0, hi = p.nseq;  // first sequence that ends after t0
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (p.off[mid + 1] <= t0) lo = mid + 1;
                else hi = mid;
            }
            int i = lo;
#pragma unroll
            for (int j = 0; j < kL; ++j) {
                const long t = t0 + j;
                while (i < p.nseq && p.off[i + 1] <= t) ++i;
                const bool ok = i < p.nseq && t < p.T && p.off[i] <= t;
                seq[j] = ok ? i : 0;
                in |= (unsigned)ok << j;
                first |= (unsigned)(ok && p.off[i] == t) << j;
                last |= (unsigned)(ok && p.off[i + 1] == t + 1) << j;
            }
        } else {
            const long n = p.T - t0;
            in = n >= kL ? (1u << kL) - 1 : (n > 0 ? (1u << n) - 1 : 0);
            seq[0] = b;
        }
    }
};

struct Shared {
    float A[kWaves][kLR * 8], U[kWaves][kLR * 8];  // a wave's composed map, per channel
    int cut[kWaves];                               // it holds a border of sequences
    float carry[2][kLR * 8];
};

// Composes the strands of a workgroup: on entry (A, U) is the lane's own map, on return `h`
// is the state that enters the lane's strand when `carry` (shared, slot `slot`) enters the
// block.  REV: the strands are taken from the last to the first.  A strand with a border of
// sequences (`cut`) lets nothing of what enters it through: a flag and not A = 0, which would
// turn an infinity of one sequence into a NaN of the next.
template <int V, bool REV, bool PACKED>
__device__ __forceinline__ void enter(Shared &sh, int slot, int waves, float (&A)[V], float (&U)[V], bool cut, float (&h)[V]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, cl = (lane & (kLR - 1)) * V;
    const int strand = REV ? 63 / kLR - lane / kLR : lane / kLR;
    // inclusive over the wave's strands
#pragma unroll
    for (int s = 1; s < 64 / kLR; s <<= 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float a = REV ? __shfl_down(A[v], s * kLR) : __shfl_up(A[v], s * kLR);
            const float u = REV ? __shfl_down(U[v], s * kLR) : __shfl_up(U[v], s * kLR);
            if (strand >= s && !(PACKED && cut)) {
                U[v] = fmaf(A[v], u, U[v]);
                A[v] *= a;
            }
        }
        if (PACKED) {
            const int c = REV ? __shfl_down((int)cut, s * kLR) : __shfl_up((int)cut, s * kLR);
            if (strand >= s) cut = cut || c;
        }
    }
    if (strand == 64 / kLR - 1) {
        if (PACKED) sh.cut[wave] = cut;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            sh.A[wave][cl + v] = A[v];
            sh.U[wave][cl + v] = U[v];
        }
    }
    __syncthreads();
    const int before = PACKED ? (REV ? __shfl_down((int)cut, kLR) : __shfl_up((int)cut, kLR)) : 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float c = sh.carry[slot][cl + v];
        for (int i = 0; i < (REV ? waves - 1 - wave : wave); ++i) {
            const int w = REV ? waves - 1 - i : i;
            c = PACKED && sh.cut[w] ? sh.U[w][cl + v] : fmaf(sh.A[w][cl + v], c, sh.U[w][cl + v]);
        }
        // exclusive: the map of the strands before this one
        const float a = REV ? __shfl_down(A[v], kLR) : __shfl_up(A[v], kLR);
        const float u = REV ? __shfl_down(U[v], kLR) : __shfl_up(U[v], kLR);
        h[v] = strand ? (PACKED && before ? u : fmaf(a, c, u)) : c;
    }
}

template <bool IOB, bool GB, bool BETA, bool PACKED, int V>
__global__ void __launch_bounds__(kThreads) scan_fwd_kernel(ScanParams p) {
    __shared__ Shared sh;
    const int waves = blockDim.x >> 6, tiles = (p.D + kLR * V - 1) / (kLR * V);
    const int b = blockIdx.x / tiles, tile = blockIdx.x % tiles;
    const int lr = threadIdx.x & (kLR - 1), strand = threadIdx.x / kLR;
    const int ch = (tile * kLR + lr) * V, n = max(0, min(V, p.D - ch));
    const bool tail = strand == waves * (64 / kLR) - 1;  // holds the block's last tokens
    if (strand == 0) {
        float c[V];
        load_state<V>(PACKED || !p.S0 ? nullptr : p.S0 + (int64_t)b * p.D + ch, n, c);
#pragma unroll
        for (int v = 0; v < V; ++v) sh.carry[0][lr * V + v] = c[v];
    }
    if (PACKED && p.ST) {  // empty sequences end as they begin
        for (int i = strand; i < p.nseq; i += waves * (64 / kLR)) {
            if (p.off[i + 1] > p.off[i]) continue;
            float c[V];
            load_state<V>(p.S0 ? p.S0 + (int64_t)i * p.D + ch : nullptr, n, c);
            store_state<V>(p.ST + (int64_t)i * p.D + ch, n, c);
        }
    }
    float h[V];
    for (int k = 0; k < p.nblk; ++k) {
        const long t0 = (long)k * kBlk + strand * kL, row = (long)b * p.T + t0;
        Marks<PACKED> m;
        m.find(p, b, t0);
        Pack<IOB, V> x[kL];
        Pack<GB, V> al[kL], be[BETA ? kL : 1];
#pragma unroll
        for (int j = 0; j < kL; ++j) {
            x[j].clear();
            al[j].clear();
            if (BETA) be[j].clear();
            if (!(m.in >> j & 1)) continue;
            x[j].load(p.x, (row + j) * p.ldx + ch, n);
            al[j].load(p.alpha, (row + j) * p.lda + ch, n);
            if (BETA) be[j].load(p.beta, (row + j) * p.ldb + ch, n);
        }
        float A[V], U[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            A[v] = 1.f;
            U[v] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < kL; ++j) {
            if (!(m.in >> j & 1)) continue;
            float s0[V];
            const bool first = PACKED && (m.first >> j & 1);
            if (first) load_state<V>(p.S0 ? p.S0 + (int64_t)m.seq[PACKED ? j : 0] * p.D + ch : nullptr, n, s0);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float a, bb;
                gates<BETA>(p, al[j].get(v), BETA ? be[BETA ? j : 0].get(v) : 0.f, a, bb);
                const float u = bb * x[j].get(v);
                if (first) {
                    U[v] = fmaf(a, s0[v], u);
                    A[v] = 0.f;
                } else {
                    U[v] = fmaf(a, U[v], u);
                    A[v] *= a;
                }
            }
        }
        enter<V, false, PACKED>(sh, k & 1, waves, A, U, m.first != 0, h);
#pragma unroll
        for (int j = 0; j < kL; ++j) {
            if (!(m.in >> j & 1)) continue;
            if (PACKED && (m.first >> j & 1))
                load_state<V>(p.S0 ? p.S0 + (int64_t)m.seq[PACKED ? j : 0] * p.D + ch : nullptr, n, h);
#pragma unroll
            for (int v = 0; v < V; v += 2) {
#pragma unroll
                for (int e = v; e < v + 2; ++e) {
                    float a, bb;
                    gates<BETA>(p, al[j].get(e), BETA ? be[BETA ? j : 0].get(e) : 0.f, a, bb);
                    h[e] = fmaf(a, h[e], bb * x[j].get(e));
                }
                x[j].set2(v, h[v], h[v + 1]);
            }
            x[j].store(p.y, (row + j) * p.D + ch, n);
            if (PACKED && p.ST && (m.last >> j & 1)) store_state<V>(p.ST + (int64_t)m.seq[PACKED ? j : 0] * p.D + ch, n, h);
        }
        if (tail) {
            if (p.ckpt) store_state<V>(p.ckpt + ((int64_t)b * p.nblk + k) * p.D + ch, n, h);
#pragma unroll
            for (int v = 0; v < V; ++v) sh.carry[(k + 1) & 1][lr * V + v] = h[v];
        }
        __syncthreads();  // the carry is written and this block's maps are read
    }
    if (!PACKED && tail && p.ST) store_state<V>(p.ST + (int64_t)b * p.D + ch, n, h);
}

template <bool IOB, bool GB, bool BETA, bool PACKED, int V>
__global__ void __launch_bounds__(kThreads) scan_bwd_kernel(ScanParams p) {
    __shared__ Shared sh, sg;
    const int waves = blockDim.x >> 6, tiles = (p.D + kLR * V - 1) / (kLR * V);
    const int b = blockIdx.x / tiles, tile = blockIdx.x % tiles;
    const int lr = threadIdx.x & (kLR - 1), strand = threadIdx.x / kLR;
    const int ch = (tile * kLR + lr) * V, n = max(0, min(V, p.D - ch));
    if (strand == 0) {
        float c[V];
        load_state<V>(PACKED || !p.dST ? nullptr : p.dST + (int64_t)b * p.D + ch, n, c);
#pragma unroll
        for (int v = 0; v < V; ++v) sg.carry[0][lr * V + v] = c[v];
    }
    if (PACKED && p.dS0) {
        for (int i = strand; i < p.nseq; i += waves * (64 / kLR)) {
            if (p.off[i + 1] > p.off[i]) continue;
            float c[V];
            load_state<V>(p.dST ? p.dST + (int64_t)i * p.D + ch : nullptr, n, c);
            store_state<V>(p.dS0 + (int64_t)i * p.D + ch, n, c);
        }
    }
    float G[V];
    for (int step = 0; step < p.nblk; ++step) {
        const int k = p.nblk - 1 - step;
        const long t0 = (long)k * kBlk + strand * kL, row = (long)b * p.T + t0;
        Marks<PACKED> m;
        m.find(p, b, t0);
        Pack<IOB, V> x[kL], dy[kL];
        Pack<GB, V> al[kL], be[BETA ? kL : 1];
#pragma unroll
        for (int j = 0; j < kL; ++j) {
            x[j].clear();
            dy[j].clear();
            al[j].clear();
            if (BETA) be[j].clear();
            if (!(m.in >> j & 1)) continue;
            x[j].load(p.x, (row + j) * p.ldx + ch, n);
            dy[j].load(p.dy, (row + j) * p.D + ch, n);
            al[j].load(p.alpha, (row + j) * p.lda + ch, n);
            if (BETA) be[j].load(p.beta, (row + j) * p.ldb + ch, n);
        }
        if (strand == 0) {  // the state that enters the block
            float c[V];
            load_state<V>(k > 0 ? p.ckpt + ((int64_t)b * p.nblk + k - 1) * p.D + ch
                                : (PACKED || !p.S0 ? nullptr : p.S0 + (int64_t)b * p.D + ch), n, c);
#pragma unroll
            for (int v = 0; v < V; ++v) sh.carry[0][lr * V + v] = c[v];
        }
        float A[V], U[V], GA[V], GU[V], h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            A[v] = GA[v] = 1.f;
            U[v] = GU[v] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < kL; ++j) {
            if (!(m.in >> j & 1)) continue;
            float s0[V];
            const bool first = PACKED && (m.first >> j & 1);
            if (first) load_state<V>(p.S0 ? p.S0 + (int64_t)m.seq[PACKED ? j : 0] * p.D + ch : nullptr, n, s0);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float a, bb;
                gates<BETA>(p, al[j].get(v), BETA ? be[BETA ? j : 0].get(v) : 0.f, a, bb);
                const float u = bb * x[j].get(v);
                if (first) {
                    U[v] = fmaf(a, s0[v], u);
                    A[v] = 0.f;
                } else {
                    U[v] = fmaf(a, U[v], u);
                    A[v] *= a;
                }
            }
        }
#pragma unroll
        for (int j = kL - 1; j >= 0; --j) {
            if (!(m.in >> j & 1)) continue;
            float st[V];
            const bool last = PACKED && (m.last >> j & 1);
            if (last) load_state<V>(p.dST ? p.dST + (int64_t)m.seq[PACKED ? j : 0] * p.D + ch : nullptr, n, st);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float a, bb;
                gates<BETA>(p, al[j].get(v), 0.f, a, bb);
                if (last) {
                    GU[v] = a * (dy[j].get(v) + st[v]);
                    GA[v] = 0.f;
                } else {
                    GU[v] = a * (dy[j].get(v) + GU[v]);
                    GA[v] *= a;
                }
            }
        }
        enter<V, false, PACKED>(sh, 0, waves, A, U, m.first != 0, h);
        enter<V, true, PACKED>(sg, step & 1, waves, GA, GU, m.last != 0, G);
        // two channels at a time: the states before each token, then the gradients from the last token back
#pragma unroll
        for (int v = 0; v < V; v += 2) {
            float before[2][kL];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float s = h[v + e];
#pragma unroll
                for (int j = 0; j < kL; ++j) {
                    before[e][j] = 0.f;
                    if (!(m.in >> j & 1)) continue;
                    if (PACKED && (m.first >> j & 1))
                        s = p.S0 && v + e < n ? p.S0[(int64_t)m.seq[PACKED ? j : 0] * p.D + ch + v + e] : 0.f;
                    before[e][j] = s;
                    float a, bb;
                    gates<BETA>(p, al[j].get(v + e), BETA ? be[BETA ? j : 0].get(v + e) : 0.f, a, bb);
                    s = fmaf(a, s, bb * x[j].get(v + e));
                }
            }
#pragma unroll
            for (int j = kL - 1; j >= 0; --j) {
                if (!(m.in >> j & 1)) continue;
                float dx[2], da[2], db[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float a, bb;
                    gates<BETA>(p, al[j].get(v + e), BETA ? be[BETA ? j : 0].get(v + e) : 0.f, a, bb);
                    if (PACKED && (m.last >> j & 1))
                        G[v + e] = p.dST && v + e < n ? p.dST[(int64_t)m.seq[PACKED ? j : 0] * p.D + ch + v + e] : 0.f;
                    const float g = dy[j].get(v + e) + G[v + e], xv = x[j].get(v + e);
                    dx[e] = bb * g;
                    db[e] = g * xv;
                    da[e] = g * (p.coupled ? before[e][j] - xv : before[e][j]);
                    if (p.log_gate) da[e] *= a;
                    G[v + e] = a * g;
                    if (PACKED && p.dS0 && (m.first >> j & 1) && v + e < n)
                        p.dS0[(int64_t)m.seq[PACKED ? j : 0] * p.D + ch + v + e] = G[v + e];
                }
                dy[j].set2(v, dx[0], dx[1]);
                al[j].set2(v, da[0], da[1]);
                if (BETA) be[BETA ? j : 0].set2(v, db[0], db[1]);
            }
        }
#pragma unroll
        for (int j = 0; j < kL; ++j) {
            if (!(m.in >> j & 1)) continue;
            dy[j].store(p.dx, (row + j) * p.D + ch, n);
            al[j].store(p.dalpha, (row + j) * p.D + ch, n);
            if (BETA) be[BETA ? j : 0].store(p.dbeta, (row + j) * p.D + ch, n);
        }
        if (strand == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) sg.carry[(step + 1) & 1][lr * V + v] = G[v];
        }
        __syncthreads();
    }
    if (!PACKED && strand == 0 && p.dS0) store_state<V>(p.dS0 + (int64_t)b * p.D + ch, n, G);
}

// One token for every batch row: the state is read and written in place.
template <bool IOB, bool GB, bool BETA, int V>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanParams p) {
    const long groups = (p.D + V - 1) / V, i = (long)blockIdx.x * 256 + threadIdx.x;
    const long b = i / groups;
    const int ch = (int)(i % groups) * V, n = min(V, p.D - ch);
    if (b >= p.B) return;
    Pack<IOB, V> x;
    Pack<GB, V> al, be;
    float *S = p.ST + b * p.D + ch;
    float h[V];
    x.load(p.x, b * p.ldx + ch, n);
    al.load(p.alpha, b * p.lda + ch, n);
    if (BETA) be.load(p.beta, b * p.ldb + ch, n);
    load_state<V>(S, n, h);
#pragma unroll
    for (int v = 0; v < V; v += 2) {
#pragma unroll
        for (int e = v; e < v + 2; ++e) {
            float a, bb;
            gates<BETA>(p, al.get(e), BETA ? be.get(e) : 0.f, a, bb);
            h[e] = fmaf(a, h[e], bb * x.get(e));
        }
        x.set2(v, h[v], h[v + 1]);
    }
    store_state<V>(S, n, h);
    x.store(p.y, b * p.D + ch, n);
}

// ST = S0 (or 0) of a call without tokens
__global__ void __launch_bounds__(256) scan_copy_kernel(const float *src, float *dst, long n) {
    const long i = (long)blockIdx.x * 256 + threadIdx.x;
    if (i < n) dst[i] = src ? src[i] : 0.f;
}

enum Kind { kFwd, kBwd, kStep };

template <Kind K, bool IOB, bool GB, bool BETA, bool PACKED, int V>
const void *kernel() {
    if constexpr (K == kFwd) return reinterpret_cast<const void *>(&scan_fwd_kernel<IOB, GB, BETA, PACKED, V>);
    if constexpr (K == kBwd) return reinterpret_cast<const void *>(&scan_bwd_kernel<IOB, GB, BETA, PACKED, V>);
    return reinterpret_cast<const void *>(&scan_step_kernel<IOB, GB, BETA, V>);
}

template <Kind K, bool IOB, bool GB>
const void *pick2(const ScanParams &p, int &v) {
    constexpr int V = IOB && GB ? 8 : 4;
    v = V;
    if (p.beta) return p.off ? kernel<K, IOB, GB, true, true, V>() : kernel<K, IOB, GB, true, false, V>();
    return p.off ? kernel<K, IOB, GB, false, true, V>() : kernel<K, IOB, GB, false, false, V>();
}

template <Kind K>
const void *pick(const ScanParams &p, int &v) {
    if (p.io_bf16) return p.gate_bf16 ? pick2<K, true, true>(p, v) : pick2<K, true, false>(p, v);
    return p.gate_bf16 ? pick2<K, false, true>(p, v) : pick2<K, false, false>(p, v);
}

hipError_t copy_states(const float *src, float *dst, long n, hipStream_t s) {
    if (!dst || n == 0 || src == dst) return hipSuccess;
    void *args[] = {&src, &dst, &n};
    return hipLaunchKernel(reinterpret_cast<const void *>(&scan_copy_kernel), dim3((unsigned)((n + 255) / 256)), dim3(256),
                           args, 0, s);
}

template <Kind K>
hipError_t launch(const ScanParams &p, hipStream_t s) {
    int v = 0;
    const void *fn = pick<K>(p, v);
    const int waves = (int)(((p.T < kBlk ? p.T : kBlk) + 63) / 64);
    ScanParams q = p;
    void *args[] = {&q};
    const long blocks = (long)p.B * ((p.D + kLR * v - 1) / (kLR * v));
    if (blocks > 0x7fffffffL) return hipErrorInvalidValue;
    return hipLaunchKernel(fn, dim3((unsigned)blocks), dim3(64 * waves), args, 0, s);
}

}  // namespace

size_t scan_workspace(const ScanParams &) { return 0; }

hipError_t launch_scan_fwd(const ScanParams &p, hipStream_t s) {
    if (p.T == 0) return copy_states(p.S0, p.ST, (long)(p.off ? p.nseq : p.B) * p.D, s);
    return launch<kFwd>(p, s);
}

hipError_t launch_scan_bwd(const ScanParams &p, hipStream_t s) {
    if (p.T == 0) return copy_states(p.dST, p.dS0, (long)(p.off ? p.nseq : p.B) * p.D, s);
    return launch<kBwd>(p, s);
}

hipError_t launch_scan_step(const ScanParams &p, hipStream_t s) {
    int v = 0;
    const void *fn = pick<kStep>(p, v);
    const long threads = (long)p.B * ((p.D + v - 1) / v);
    if ((threads + 255) / 256 > 0x7fffffffL) return hipErrorInvalidValue;
    ScanParams q = p;
    void *args[] = {&q};
    return hipLaunchKernel(fn, dim3((unsigned)((threads + 255) / 256)), dim3(256), args, 0, s);
}

}  // namespace gdr
