// delta_prep.hip -- per chunk and value head of the delta rule: T = (I + A)^{-1} and the scores Q (delta.hpp),
// and k, q laid out as the operands of the chain's products.
#include "delta.hpp"
#include "gdr_ut.hpp"

namespace gdr {
namespace {

// Places (16-row tile, 32-column block) of a lower triangular matrix, and of an upper one.
__device__ __forceinline__ int tri_tile(bool upper, int i) { return upper ? (i < 2 ? 0 : i < 4 ? 1 : i - 2) : (i < 2 ? i : i < 4 ? 2 : 3); }
__device__ __forceinline__ int tri_block(bool upper, int i) { return upper ? (i < 4 ? i & 1 : 1) : (i < 2 ? 0 : i & 1); }

template <int NT, int KB, bool BWD>
__global__ void __launch_bounds__(256) delta_prep_kernel(DeltaParams p) {
    constexpr int D = 32 * KB, LD = D + 8;
    __shared__ __attribute__((aligned(16))) uint16_t Kt[NT][kDeltaC][LD];
    __shared__ __attribute__((aligned(16))) uint16_t Qt[NT][kDeltaC][LD];
    __shared__ __attribute__((aligned(16))) float As[kDeltaC][kUtN + 4];
    __shared__ __attribute__((aligned(16))) float Ps[kDeltaC][kUtN + 4];
    __shared__ float Xs[4][16][16];
    __shared__ ChunkGates gt;
    const int hv = blockIdx.x % p.Hv, slot = blockIdx.x / p.Hv, hk = hv / p.group;
    const Place at = place_of(p, slot);
    if (at.n <= 0) return;  // uniform over the workgroup
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, r = l & 15, q = l >> 4;
    for (int i = tid; i < kDeltaC * D / 8; i += 256) {
        const int row = i / (D / 8), ch = i % (D / 8) * 8;
        const bool there = row < at.n && ch < p.dk;
        bf16x8 t[NT];
        load8<NT>(p.k, (at.row0 + row) * p.ldk + (long)hk * p.dk + ch, there, t);
#pragma unroll
        for (int n = 0; n < NT; ++n) *reinterpret_cast<bf16x8 *>(&Kt[n][row][ch]) = t[n];
        load8<NT>(p.q, (at.row0 + row) * p.ldq + (long)hk * p.dk + ch, there, t);
#pragma unroll
        for (int n = 0; n < NT; ++n) *reinterpret_cast<bf16x8 *>(&Qt[n][row][ch]) = t[n];
    }
    if (w == 0) make_gates(p, at, hv, l, gt);
    __syncthreads();
    const long head = (long)slot * p.Hv + hv;
    if (w == 0) {
        float *gp = p.gates + head * kDeltaGates;
        gp[l] = gt.front[l];
        gp[64 + l] = gt.behind[l] * gt.beta[l];
        if (l == 0) gp[128] = gt.whole;
    }
    // row tile w against the column tiles up to it
    bf16x8 ak[KB][NT], aq[KB][NT];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            ak[kb][n] = *reinterpret_cast<const bf16x8 *>(&Kt[n][16 * w + r][32 * kb + 8 * q]);
            aq[kb][n] = *reinterpret_cast<const bf16x8 *>(&Qt[n][16 * w + r][32 * kb + 8 * q]);
        }
    for (int j = 0; j < 4; ++j) {
        f32x4 kk = {0.f, 0.f, 0.f, 0.f}, qk = kk;
        if (j <= w) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                bf16x8 b[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) b[n] = *reinterpret_cast<const bf16x8 *>(&Kt[n][16 * j + r][32 * kb + 8 * q]);
                kk = product<NT, NT>(ak[kb], b, kk);
                qk = product<NT, NT>(aq[kb], b, qk);
            }
        }
        const int s = 16 * j + r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 16 * w + 4 * q + i;
            const float eb = t >= s ? gt.decay(t, s) * gt.beta[s] : 0.f;
            As[t][s] = t > s ? eb * kk[i] : 0.f;
            Ps[t][s] = t >= s ? eb * qk[i] : 0.f;
        }
    }
    __syncthreads();
    ut_transform<kUtN + 4>(As, As, Xs, w, l);
    for (int i = w; i < 12; i += 4) {
        const float(*M)[kUtN + 4] = i < 6 ? As : Ps;
        const int c = i % 6, a = tri_tile(BWD, c), b = tri_block(BWD, c);
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int m = 16 * a + r, n = 32 * b + perm(q, e);
            x[e] = BWD ? M[n][m] : M[m][n];
        }
        bf16x8 t[3];
        split<3>(x, t);
        char *out = i < 6 ? p.tf : p.pf;
#pragma unroll
        for (int n = 0; n < 3; ++n) put_fragment(out, head * kDeltaTri + 3 * c + n, l, t[n]);
    }
    if (hv % p.group) return;
    const long key = (long)slot * p.Hk + hk;
    for (int i = w; i < 4 * KB * NT; i += 4) {  // k and q by rows: block kb of channels, tile a, term n
        const int n = i % NT, a = i / NT % 4, kb = i / NT / 4;
        const uint16_t *kr = &Kt[n][16 * a + r][32 * kb + 4 * q], *qr = &Qt[n][16 * a + r][32 * kb + 4 * q];
        const u32x2 k0 = *reinterpret_cast<const u32x2 *>(kr), k1 = *reinterpret_cast<const u32x2 *>(kr + 16);
        const u32x2 q0 = *reinterpret_cast<const u32x2 *>(qr), q1 = *reinterpret_cast<const u32x2 *>(qr + 16);
        put_fragment(p.kf, key * (4 * KB * NT) + i, l, as_bf16x8((u32x4){k0[0], k0[1], k1[0], k1[1]}));
        put_fragment(p.qf, key * (4 * KB * NT) + i, l, as_bf16x8((u32x4){q0[0], q0[1], q1[0], q1[1]}));
    }
    for (int i = w; i < 4 * KB * NT; i += 4) {  // and by channels: block tb of tokens, tile a of channels
        const int n = i % NT, a = i / NT % (2 * KB), tb = i / NT / (2 * KB);
        u32x4 kw, qw;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const int t0 = 32 * tb + perm(q, e), c = 16 * a + r;
            kw[e / 2] = Kt[n][t0][c] | (uint32_t)Kt[n][t0 + 1][c] << 16;
            if (BWD) qw[e / 2] = Qt[n][t0][c] | (uint32_t)Qt[n][t0 + 1][c] << 16;
        }
        put_fragment(p.ktf, key * (4 * KB * NT) + i, l, as_bf16x8(kw));
        if (BWD) put_fragment(p.qtf, key * (4 * KB * NT) + i, l, as_bf16x8(qw));
    }
}

template <bool BWD>
const void *pick(int nt, int kb) {
    if (nt == 1) return kb == 2 ? reinterpret_cast<const void *>(&delta_prep_kernel<1, 2, BWD>) : reinterpret_cast<const void *>(&delta_prep_kernel<1, 4, BWD>);
    return kb == 2 ? reinterpret_cast<const void *>(&delta_prep_kernel<3, 2, BWD>) : reinterpret_cast<const void *>(&delta_prep_kernel<3, 4, BWD>);
}

}  // namespace

size_t delta_workspace(DeltaParams &p, bool bwd, char *base) {
    size_t at = 0;
    auto take = [&](size_t n) {
        char *r = base + at;
        at += (n + 1023) / 1024 * 1024;
        return r;
    };
    const size_t nt = p.io_bf16 ? 1 : 3, key = (size_t)p.nslot * p.Hk * 4 * delta_blocks(p.dk) * nt * 1024;
    const size_t heads = (size_t)p.nslot * p.Hv;
    p.kf = take(key);
    p.ktf = take(key);
    p.qf = take(key);
    p.qtf = bwd ? take(key) : nullptr;
    p.tf = take(heads * kDeltaTri * 1024);
    p.pf = take(heads * kDeltaTri * 1024);
    p.gates = reinterpret_cast<float *>(take(heads * kDeltaGates * 4));
    p.back = bwd ? reinterpret_cast<float *>(take(heads * delta_tiles(p.dk, p.dv) * 1024)) : nullptr;
    p.sum = bwd && p.group > 1 ? reinterpret_cast<float *>(take((size_t)p.nslot * p.Hk * 16 * delta_blocks(p.dk) * 1024)) : nullptr;
    return at;
}

hipError_t launch_delta_prep(const DeltaParams &p0, bool bwd, hipStream_t s) {
    DeltaParams p = p0;
    void *args[] = {&p};
    const int nt = p.io_bf16 ? 1 : 3, kb = delta_blocks(p.dk);
    return hipLaunchKernel(bwd ? pick<true>(nt, kb) : pick<false>(nt, kb), dim3((unsigned)p.nslot * p.Hv), dim3(256), args, 0, s);
}

}  // namespace gdr
