// scan_bwd.hip -- gated linear recurrence: the backward pass (see scan_impl.hpp).
//
// Measured, back to back through the binding, so with the fill of the chain: 4 x 4,096 tokens of 2,048
// channels, log gates coupled: bf16 101 us (3.3 TB/s), bf16 with fp32 gates 114 us (4.1), fp32 138 us
// (4.9); value gates: 83 us (4.0), 102 us (4.6), 131 us (5.1); 65,536 of 2,032, value gates: bf16 356 us
// (3.7) and fp32 496 us (5.4).  Packed, 37 sequences of 20,000 x 1,000, beta: bf16 113 us (57 of data), fp32
// 159 us (114; 133 unpacked).  65,536 of 231 bf16 64 us, of 232 50 us.
// The inputs of a block and both of its decays and factors stay in registers (160 to 233), which leaves one
// workgroup to a compute unit.  Forcing two spills; forming the factors of log gates again behind the wait
// costs more than it frees (95 us to 111 and more), which was not tried with value gates, where a factor
// is a shift or a difference; nor was keeping inputs in shared memory over the wait.
#include "scan_impl.hpp"

namespace gdr {
namespace {

template <bool IOB, bool GB, int F, bool LOG, bool PACKED>
__global__ void __launch_bounds__(kThreads) scan_bwd_kernel(ScanParams p) {
    constexpr int LB = F == kGiven ? L : 1;
    __shared__ Shared sh, sg;
    __shared__ int ticket;
    const int waves = blockDim.x >> 6;
    const unsigned tiles = (p.D + CH - 1) / CH, columns = p.B * tiles, id = place(p, ticket);
    const unsigned column = id % columns, step = id / columns, k = p.nblk - 1 - step;  // from the last block to the first
    const unsigned b = column / tiles, tile = column % tiles;
    const int lr = threadIdx.x & (kLR - 1), strand = threadIdx.x / kLR;
    const int ch = (tile * kLR + lr) * V, n = max(0, min(V, p.D - ch));
    const bool whole = (tile + 1) * CH <= (unsigned)p.D || p.D % V == 0;
    const int local = strand * L, t0 = k * kBlk + local;
    const int rows = min(kBlk, p.T - (int)k * kBlk);  // of this block
    const int64_t row = (int64_t)b * p.T + k * kBlk;  // its first
    const unsigned there = rows >= local + L ? (1u << L) - 1 : rows > local ? (1u << (rows - local)) - 1 : 0;
    Pack<IOB> x[L], dy[L];
    Pack<GB> al[L], be[LB];
    Rows<IOB>(p.x, row, rows, p.ldx, p.D, local, ch).load(x, whole, n);
    Rows<GB>(p.alpha, row, rows, p.lda, p.D, local, ch).load(al, whole, n);
    if constexpr (F == kGiven) Rows<GB>(p.beta, row, rows, p.ldb, p.D, local, ch).load(be, whole, n);
    Rows<IOB>(p.dy, row, rows, p.D, p.D, local, ch).load(dy, whole, n);
    Marks<PACKED> m;
    m.find(p, t0, there);
    const States S0(p.S0, PACKED ? p.nseq : p.B, p.D, ch), dST(p.dST, PACKED ? p.nseq : p.B, p.D, ch), dS0(p.dS0, PACKED ? p.nseq : p.B, p.D, ch);
    if (PACKED && p.dS0 && k == 0) {
        for (int i = strand; i < p.nseq; i += waves * kWS) {
            if (p.off[i + 1] > p.off[i]) continue;
            float c[V];
            dST.load(i, c);
            dS0.store(i, n, c);
        }
    }
    if (PACKED || rows < kBlk) {
        leave_out<LOG>(m.in, x, al, be);
#pragma unroll
        for (int j = 0; j < L; ++j)
            dy[j].choose(m.in >> j & 1, 0);
    }
    float a[L][V], bb[L][V], A[V], U[V], GA[V], GU[V], h[V], G[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        A[v] = GA[v] = 1.f;
        U[v] = GU[v] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < L; ++j) {
        gates<F, LOG, GB>(al[j], be[j % LB], a[j], bb[j]);
        const bool first = PACKED && (m.first >> j & 1);
        if (first) S0.load(m.seq[j], U);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            U[v] = fmaf(a[j][v], U[v], bb[j][v] * x[j].get(v));
            A[v] = first ? 0.f : A[v] * a[j][v];
        }
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = L - 1; j >= 0; --j) {
        const bool end = PACKED && (m.last >> j & 1);
        if (end) dST.load(m.seq[j], GU);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            GU[v] = a[j][v] * (dy[j].get(v) + GU[v]);
            GA[v] = end ? 0.f : GA[v] * a[j][v];
        }
    }
    bool cut = m.first != 0, gcut = m.last != 0;
    compose<false, PACKED>(sh, A, U, cut);
    compose<true, PACKED>(sg, GA, GU, gcut);
    __syncthreads();
    {
        // one wave joins the chain of gradients while another one takes the kept state into the block
        const int c = threadIdx.x & 63, cc = tile * CH + c, wave = threadIdx.x >> 6;
        if (wave == 0) {
            const Map own = block_map<true, PACKED>(sg, waves, c);
            float in = !PACKED && step == 0 && p.dST && cc < p.D ? p.dST[(int64_t)b * p.D + cc] : 0.f, out;
            if (p.nblk > 1) in = Chain<kGroupBwd>(p, column, c).join(step, own, in, out);
            wave_states<true, PACKED>(sg, waves, c, in);
        }
        if (wave == (waves > 1 ? 1 : 0)) {
            float in = 0.f;
            if (cc < p.D) {
                if (k > 0) in = p.ckpt[((int64_t)b * p.nblk + k - 1) * p.D + cc];
                else if (!PACKED && p.S0) in = p.S0[(int64_t)b * p.D + cc];
            }
            wave_states<false, PACKED>(sh, waves, c, in);
        }
    }
    __syncthreads();
    strand_states<false, PACKED>(sh, A, U, cut, h);
    strand_states<true, PACKED>(sg, GA, GU, gcut, G);
    // two channels at a time: the states before each token, then the gradients from the last token back
#pragma unroll
    for (int v = 0; v < V; v += 2) {
        float before[2][L];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float s = h[v + e];
#pragma unroll
            for (int j = 0; j < L; ++j) {
                if (PACKED && (m.first >> j & 1)) s = S0.load1(m.seq[j], v + e);
                before[e][j] = s;
                s = fmaf(a[j][v + e], s, bb[j][v + e] * x[j].get(v + e));
            }
        }
#pragma unroll
        for (int j = L - 1; j >= 0; --j) {
            float dx[2], da[2], db[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (PACKED && (m.last >> j & 1)) G[v + e] = dST.load1(m.seq[j], v + e);
                const float g = dy[j].get(v + e) + G[v + e], xv = x[j].get(v + e);
                dx[e] = bb[j][v + e] * g;
                db[e] = g * xv;
                G[v + e] = a[j][v + e] * g;
                da[e] = (LOG ? G[v + e] : g) * (F == kCoupled ? before[e][j] - xv : before[e][j]);
                if (PACKED && (m.first >> j & 1)) dS0.store1(m.seq[j], v + e, n, G[v + e]);
            }
            dy[j].set2(v, dx[0], dx[1]);
            al[j].set2(v, da[0], da[1]);
            if (F == kGiven) be[j % LB].set2(v, db[0], db[1]);
        }
    }
    Rows<IOB>(p.dx, row, rows, p.D, p.D, local, ch).store(dy, m.in, whole, n);
    Rows<GB>(p.dalpha, row, rows, p.D, p.D, local, ch).store(al, m.in, whole, n);
    if constexpr (F == kGiven) Rows<GB>(p.dbeta, row, rows, p.D, p.D, local, ch).store(be, m.in, whole, n);
    if (!PACKED && strand == 0 && k == 0) dS0.store(b, n, G);
}

struct Bwd {
    static int group(const ScanParams &) { return kGroupBwd; }
    template <bool IOB, bool GB, int F, bool LOG, bool PACKED>
    static const void *get() { return reinterpret_cast<const void *>(&scan_bwd_kernel<IOB, GB, F, LOG, PACKED>); }
};

}  // namespace

hipError_t launch_scan_bwd(const ScanParams &p, hipStream_t s) {
    if (p.T == 0) return launch_scan_copy(p.dST, p.dS0, (long)(p.off ? p.nseq : p.B) * p.D, s);
    return launch_blocks<Bwd>(p, s);
}

}  // namespace gdr
