// delta_chain.hip -- the recurrence of the delta rule over a sequence's chunks, forward and backward (delta.hpp).
#include "delta.hpp"

namespace gdr {
namespace {

template <int NT>
__device__ __forceinline__ void fragments(const char *base, long at, int lane, bf16x8 (&t)[NT]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) t[n] = fragment(base, at + n, lane);
}

// Places (16-row tile, 32-column block) of triangular operands: i counts the six that are not zero.
template <bool UPPER>
constexpr int tri_index(int a, int b) {
    return UPPER ? (a < 2 ? 2 * a + b : b == 1 ? a + 2 : -1) : (a < 2 ? (b == 0 ? a : -1) : 2 * a - 2 + b);
}

// One wave has 16 columns of one value head's state, all of its rows, in registers.  Nothing is
// exchanged: every product's result is the next one's operand as it lies (perm in delta.hpp).
template <int NT, int KB, bool BWD>
__global__ void __launch_bounds__(64) delta_chain_kernel(DeltaParams p, int heads8) {
    constexpr int NX = NT == 1 ? 2 : 3;  // terms of what only outputs of the io type read
    const int head = blockIdx.x % heads8, tile = blockIdx.x / heads8;
    if (head >= p.nseq * p.Hv) return;
    const int seq = head / p.Hv, hv = head % p.Hv, hk = hv / p.group;
    const int l = threadIdx.x, r = l & 15, q = l >> 4, col = 16 * tile + r;
    const bool mine = col < p.dv;
    long row0;
    const int len = tokens_of(p, seq, row0), nc = (len + kDeltaC - 1) / kDeltaC;
    const int slot0 = first_slot(p, seq);
    const long sstate = (long)p.dk * p.dv, sckpt = sstate + (long)kDeltaC * p.dv;
    f32x4 S[2 * KB];
    const float *init = BWD ? p.dST : p.S0;
#pragma unroll
    for (int a = 0; a < 2 * KB; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ch = 16 * a + 4 * q + i;
            S[a][i] = init && mine && ch < p.dk ? init[head * sstate + (long)ch * p.dv + col] : 0.f;
        }
    auto keep = [&](float *to) __attribute__((always_inline)) {
#pragma unroll
        for (int a = 0; a < 2 * KB; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int ch = 16 * a + 4 * q + i;
                if (mine && ch < p.dk) to[(long)ch * p.dv + col] = S[a][i];
            }
    };
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    for (int cc = 0; cc < nc; ++cc) {
        const int c = BWD ? nc - 1 - cc : cc;
        const int n = min(kDeltaC, len - c * kDeltaC);
        const long slot = slot0 + c, vh = slot * p.Hv + hv, kh = slot * p.Hk + hk;
        const long row = row0 + (long)c * kDeltaC;
        const float *gates = p.gates + vh * kDeltaGates;
        const long kbase = kh * (4 * KB * NT), tbase = vh * kDeltaTri;
        if constexpr (BWD) keep(p.G + vh * sstate);
        else if (p.ckpt) keep(p.ckpt + vh * sckpt);
        // v, or do, of the lane's rows 16 a + 4 q + i
        f32x4 x[4];
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 16 * a + 4 * q + i;
                const long at = BWD ? ((row + t) * p.Hv + hv) * p.dv + col : (row + t) * p.ldv + (long)hv * p.dv + col;
                x[a][i] = mine && t < n ? ld_elem(BWD ? p.dout : p.v, at, NT == 1) : 0.f;
            }
        f32x4 front[4], wb[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            front[a] = *reinterpret_cast<const f32x4 *>(gates + 16 * a + 4 * q);
            wb[a] = *reinterpret_cast<const f32x4 *>(gates + 64 + 16 * a + 4 * q);
        }
        const float whole = gates[128];
        f32x4 R[4] = {zero, zero, zero, zero}, O[4] = {zero, zero, zero, zero};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            bf16x8 sf[3];
            split<3>(S[2 * kb], S[2 * kb + 1], sf);
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                bf16x8 kf[NT];
                fragments<NT>(p.kf, kbase + (a * KB + kb) * NT, l, kf);
                R[a] = product<NT, 3>(kf, sf, R[a]);
            }
            if constexpr (!BWD) {
                bf16x8 sx[NX];
#pragma unroll
                for (int m = 0; m < NX; ++m) sx[m] = sf[m];
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    bf16x8 qf[NT];
                    fragments<NT>(p.qf, kbase + (a * KB + kb) * NT, l, qf);
                    O[a] = product<NT, NX>(qf, sx, O[a]);
                }
            }
        }
        f32x4 E[4] = {zero, zero, zero, zero};
        if constexpr (!BWD) {
            // E = T (v - front k S), o = front q S + Q E
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                R[a] = x[a] - front[a] * R[a];
                O[a] = front[a] * O[a];
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                bf16x8 rf[3];
                split<3>(R[2 * b], R[2 * b + 1], rf);
#pragma unroll
                for (int a = 2 * b; a < 4; ++a) {
                    bf16x8 tf[3];
                    fragments<3>(p.tf, tbase + 3 * tri_index<false>(a, b), l, tf);
                    E[a] = product<3, 3>(tf, rf, E[a]);
                }
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                bf16x8 ef[NX];
                split<NX>(E[2 * b], E[2 * b + 1], ef);
#pragma unroll
                for (int a = 2 * b; a < 4; ++a) {
                    bf16x8 pf[NX];
                    fragments<NX>(p.pf, tbase + 3 * tri_index<false>(a, b), l, pf);
                    O[a] = product<NX, NX>(pf, ef, O[a]);
                }
            }
        } else {
            // E = T^T (Q^T do + wb k G)
#pragma unroll
            for (int a = 0; a < 4; ++a) R[a] = wb[a] * R[a];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                bf16x8 df[NT];
                split<NT>(x[2 * b], x[2 * b + 1], df);
#pragma unroll
                for (int a = 0; a < 2 + 2 * b; ++a) {
                    bf16x8 pf[3];
                    fragments<3>(p.pf, tbase + 3 * tri_index<true>(a, b), l, pf);
                    R[a] = product<3, NT>(pf, df, R[a]);
                }
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                bf16x8 rf[3];
                split<3>(R[2 * b], R[2 * b + 1], rf);
#pragma unroll
                for (int a = 0; a < 2 + 2 * b; ++a) {
                    bf16x8 tf[3];
                    fragments<3>(p.tf, tbase + 3 * tri_index<true>(a, b), l, tf);
                    E[a] = product<3, 3>(tf, rf, E[a]);
                }
            }
        }
        // S = whole S + k^T (wb E), or whole S + q^T (front do) - k^T (front E)
#pragma unroll
        for (int a = 0; a < 2 * KB; ++a) S[a] = whole * S[a];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            bf16x8 ef[3];
            if constexpr (BWD) split<3>(-front[2 * b] * E[2 * b], -front[2 * b + 1] * E[2 * b + 1], ef);
            else split<3>(wb[2 * b] * E[2 * b], wb[2 * b + 1] * E[2 * b + 1], ef);
#pragma unroll
            for (int a = 0; a < 2 * KB; ++a) {
                bf16x8 kt[NT];
                fragments<NT>(p.ktf, kbase + (a * 2 + b) * NT, l, kt);
                S[a] = product<NT, 3>(kt, ef, S[a]);
            }
            if constexpr (BWD) {
                bf16x8 df[3];
                split<3>(front[2 * b] * x[2 * b], front[2 * b + 1] * x[2 * b + 1], df);
#pragma unroll
                for (int a = 0; a < 2 * KB; ++a) {
                    bf16x8 qt[NT];
                    fragments<NT>(p.qtf, kbase + (a * 2 + b) * NT, l, qt);
                    S[a] = product<NT, 3>(qt, df, S[a]);
                }
            }
        }
        float *Et = BWD ? p.y + vh * ((long)kDeltaC * p.dv) : p.ckpt ? p.ckpt + vh * sckpt + sstate : nullptr;
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 16 * a + 4 * q + i;
                if (!mine) continue;
                if (Et) Et[(long)t * p.dv + col] = E[a][i];
                if (t < n) st_elem(BWD ? p.dvv : p.o, ((row + t) * p.Hv + hv) * p.dv + col, BWD ? E[a][i] : O[a][i], NT == 1);
            }
    }
    float *last = BWD ? p.dS0 : p.ST;
    if (last) keep(last + head * sstate);
}

template <bool BWD>
const void *pick(int nt, int kb) {
    if (nt == 1) return kb == 2 ? reinterpret_cast<const void *>(&delta_chain_kernel<1, 2, BWD>) : reinterpret_cast<const void *>(&delta_chain_kernel<1, 4, BWD>);
    return kb == 2 ? reinterpret_cast<const void *>(&delta_chain_kernel<3, 2, BWD>) : reinterpret_cast<const void *>(&delta_chain_kernel<3, 4, BWD>);
}

// Heads of the grid: a multiple of 8, so that the column tiles of one head run on one of the 8 XCDs
// (workgroups go round them in turn) and share its operands in that one's cache.
long heads_of(const DeltaParams &p) { return ((long)p.nseq * p.Hv + 7) / 8 * 8; }

}  // namespace

hipError_t launch_delta_chain(const DeltaParams &p0, bool bwd, hipStream_t s) {
    DeltaParams p = p0;
    int heads = (int)heads_of(p);
    void *args[] = {&p, &heads};
    const int nt = p.io_bf16 ? 1 : 3, kb = delta_blocks(p.dk);
    return hipLaunchKernel(bwd ? pick<true>(nt, kb) : pick<false>(nt, kb), dim3((unsigned)heads * ((p.dv + 15) / 16)), dim3(64), args, 0, s);
}

hipError_t launch_delta_fwd(const DeltaParams &p, hipStream_t s) {
    hipError_t e = p.nslot > 0 ? launch_delta_prep(p, false, s) : hipSuccess;
    return e == hipSuccess ? launch_delta_chain(p, false, s) : e;
}

hipError_t launch_delta_bwd(const DeltaParams &p, hipStream_t s) {
    hipError_t e = p.nslot > 0 ? launch_delta_prep(p, true, s) : hipSuccess;
    if (e == hipSuccess) e = launch_delta_chain(p, true, s);
    return e == hipSuccess && p.nslot > 0 ? launch_delta_grad(p, s) : e;
}

}  // namespace gdr
