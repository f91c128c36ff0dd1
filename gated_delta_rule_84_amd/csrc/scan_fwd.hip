// scan_fwd.hip -- gated linear recurrence: the forward pass (see scan_impl.hpp).
//
// Measured, back to back through the binding, so with the fill of the chain: 4 x 4,096 tokens of 2,048
// channels, log gates coupled: bf16 50 us (4.0 TB/s), bf16 with fp32 gates 56 to 62 us (4.3 to 4.8), fp32
// 86 us (4.7); 65,536 of 2,032 bf16 202 us (4.0) and fp32 298 us (5.4).  Bound by the chain: 65,536 of 128
// bf16 29 us (10 us of data), 400,000 of 40 bf16 79 us (20).  Packed, 37 sequences of 20,000 x 1,000, beta:
// fp32 96 to 103 us (65 of data; 74 unpacked), bf16 66 us (33).  Channels whose number is not a multiple of
// 4 go element by element in the last tile: 65,536 of 231 bf16 42 us, of 232 35 us.
// 128 registers (launch bounds of 4 waves per SIMD) keep two workgroups on a compute unit, so that
// one loads while the other waits for the chain.
#include "scan_impl.hpp"

namespace gdr {
namespace {

template <bool IOB, bool GB, int F, bool LOG, bool PACKED>
__global__ void __launch_bounds__(kThreads, 4) scan_fwd_kernel(ScanParams p) {
    constexpr int LB = F == kGiven ? L : 1;
    __shared__ Shared sh;
    __shared__ int ticket;
    const int waves = blockDim.x >> 6;
    const unsigned tiles = (p.D + CH - 1) / CH, columns = p.B * tiles, id = place(p, ticket);
    const unsigned column = id % columns, k = id / columns, b = column / tiles, tile = column % tiles;
    const int lr = threadIdx.x & (kLR - 1), strand = threadIdx.x / kLR;
    const int ch = (tile * kLR + lr) * V, n = max(0, min(V, p.D - ch));
    const bool whole = (tile + 1) * CH <= (unsigned)p.D || p.D % V == 0;  // no lane's channels end inside
    const int local = strand * L, t0 = k * kBlk + local;
    const int rows = min(kBlk, p.T - (int)k * kBlk);  // of this block
    const int64_t row = (int64_t)b * p.T + k * kBlk;  // its first
    const unsigned there = rows >= local + L ? (1u << L) - 1 : rows > local ? (1u << (rows - local)) - 1 : 0;
    Pack<IOB> x[L];
    Pack<GB> al[L], be[LB];
    Rows<IOB>(p.x, row, rows, p.ldx, p.D, local, ch).load(x, whole, n);
    Rows<GB>(p.alpha, row, rows, p.lda, p.D, local, ch).load(al, whole, n);
    if constexpr (F == kGiven) Rows<GB>(p.beta, row, rows, p.ldb, p.D, local, ch).load(be, whole, n);
    Marks<PACKED> m;
    m.find(p, t0, there);
    const States S0(p.S0, PACKED ? p.nseq : p.B, p.D, ch), ST(p.ST, PACKED ? p.nseq : p.B, p.D, ch);
    if (PACKED && p.ST && k == 0) {  // empty sequences end as they begin
        for (int i = strand; i < p.nseq; i += waves * kWS) {
            if (p.off[i + 1] > p.off[i]) continue;
            float c[V];
            S0.load(i, c);
            ST.store(i, n, c);
        }
    }
    if (PACKED || rows < kBlk) leave_out<LOG>(m.in, x, al, be);
    float a[L][V], u[L][V], A[V], U[V], h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        A[v] = 1.f;
        U[v] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < L; ++j) {
        gates<F, LOG, GB>(al[j], be[j % LB], a[j], u[j]);
        const bool first = PACKED && (m.first >> j & 1);
        if (first) S0.load(m.seq[j], U);
#pragma unroll
        for (int v = 0; v < V; ++v) u[j][v] *= x[j].get(v);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            U[v] = fmaf(a[j][v], U[v], u[j][v]);
            A[v] = first ? 0.f : A[v] * a[j][v];
        }
        __builtin_amdgcn_sched_barrier(0);  // a token at a time, or the exponentials of all are in flight at once
    }
    bool cut = m.first != 0;
    compose<false, PACKED>(sh, A, U, cut);
    __syncthreads();
    if (threadIdx.x < CH) {
        const int c = threadIdx.x, cc = tile * CH + c;
        const Map own = block_map<false, PACKED>(sh, waves, c);
        float in = !PACKED && k == 0 && p.S0 && cc < p.D ? p.S0[(int64_t)b * p.D + cc] : 0.f, out = own.apply(in);
        if (p.nblk > 1) in = Chain<PACKED ? kGroupPacked : kGroupFwd>(p, column, c).join(k, own, in, out);
        wave_states<false, PACKED>(sh, waves, c, in);
        if (p.ckpt && cc < p.D) p.ckpt[((int64_t)b * p.nblk + k) * p.D + cc] = out;
    }
    __syncthreads();
    strand_states<false, PACKED>(sh, A, U, cut, h);
#pragma unroll
    for (int j = 0; j < L; ++j) {
        if (PACKED && (m.first >> j & 1)) S0.load(m.seq[j], h);
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = fmaf(a[j][v], h[v], u[j][v]);
#pragma unroll
        for (int v = 0; v < V; v += 2) x[j].set2(v, h[v], h[v + 1]);
        if (PACKED && (m.last >> j & 1)) ST.store(m.seq[j], n, h);
    }
    Rows<IOB>(p.y, row, rows, p.D, p.D, local, ch).store(x, m.in, whole, n);
    if (!PACKED && k == p.nblk - 1 && strand == waves * kWS - 1) ST.store(b, n, h);
}

struct Fwd {
    static int group(const ScanParams &p) { return p.off ? kGroupPacked : kGroupFwd; }
    template <bool IOB, bool GB, int F, bool LOG, bool PACKED>
    static const void *get() { return reinterpret_cast<const void *>(&scan_fwd_kernel<IOB, GB, F, LOG, PACKED>); }
};

}  // namespace

hipError_t launch_scan_fwd(const ScanParams &p, hipStream_t s) {
    if (p.T == 0) return launch_scan_copy(p.S0, p.ST, (long)(p.off ? p.nseq : p.B) * p.D, s);
    return launch_blocks<Fwd>(p, s);
}

}  // namespace gdr
