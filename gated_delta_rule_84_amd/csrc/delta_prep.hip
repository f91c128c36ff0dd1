// delta_prep.hip -- per chunk and value head of the delta rule: T = (I + A)^{-1} and the scores Q (delta.hpp),
// and k, q laid out as the operands of the chain's products.
#include "delta.hpp"
#include "gdr_ut.hpp"

namespace gdr {
namespace {

// Places (16-row tile, 32-column block) of a lower triangular matrix, and of an upper one.
__device__ __forceinline__ int tri_tile(bool upper, int i) { return upper ? (i < 2 ? 0 : i < 4 ? 1 : i - 2) : (i < 2 ? i : i < 4 ? 2 : 3); }
__device__ __forceinline__ int tri_block(bool upper, int i) { return upper ? (i < 4 ? i & 1 : 1) : (i < 2 ? 0 : i & 1); }

// A workgroup per chunk and value head: four waves, a tile of 16 tokens each.  k lies in shared memory, which every pair of
// tiles reads; q is read by its own wave only and stays in registers.  Bound by the inverse's dependent steps and the workgroup's loads:
// 4 x 4,096 tokens, 16 heads of 128, bf16, 61 us, for the backward pass (which needs 3 terms of Q) 86; 0.28 and 0.3 GB moved.
template <int NT, int KB, bool BWD>
__global__ void __launch_bounds__(256) delta_prep_kernel(DeltaParams p) {
    constexpr int D = 32 * KB;
    __shared__ __attribute__((aligned(16))) Staged<D, NT, kDeltaC> k;
    __shared__ __attribute__((aligned(16))) float As[kDeltaC][kUtN + 4];
    __shared__ float Xs[4][16][16];
    __shared__ ChunkGates gt;
    const int hv = blockIdx.x % p.Hv, slot = blockIdx.x / p.Hv, hk = hv / p.group;
    const Place at = place_of(p, slot);
    if (at.n <= 0) return;  // uniform over the workgroup
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, r = l & 15, q = l >> 4;
    constexpr int kPieces = kDeltaC * D / 8 / 256;
    {
        bf16x8 t[kPieces][NT];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int row = (tid + 256 * i) / (D / 8), m = (tid + 256 * i) % (D / 8);
            load8<NT>(p.k, (at.row0 + row) * p.ldk + (long)hk * p.dk + 8 * m, row < at.n && 8 * m < p.dk, t[i]);
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) k.put8((tid + 256 * i) / (D / 8), (tid + 256 * i) % (D / 8), t[i]);
    }
    if (w == 0) make_gates(p, at, hv, l, gt);
    // this wave's places of the scores, a tile of rows (forward t, backward s) and a block of columns, and q of their tokens
    constexpr int kMine = 2;  // the second only for waves 0 and 1
    bf16x8 qf[kMine][BWD ? 2 : 1][KB][NT];
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
        const int c = w + 4 * m, a = tri_tile(BWD, c), b = tri_block(BWD, c);
#pragma unroll
        for (int z = 0; z < (BWD ? 2 : 1); ++z) {
            const int row = 16 * (BWD ? 2 * b + z : a) + r;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
                load8<NT>(p.q, (at.row0 + row) * p.ldq + (long)hk * p.dk + 32 * kb + 8 * q, c < 6 && row < at.n && 32 * kb + 8 * q < p.dk,
                          qf[m][z][kb]);
        }
    }
    __syncthreads();
    const long head = (long)slot * p.Hv + hv;
    if (w == 0) {
        float *gp = p.gates + head * kDeltaGates;
        gp[l] = gt.front[l];
        gp[64 + l] = gt.behind[l] * gt.beta[l];
        if (l == 0) gp[128] = gt.whole;
    }
    // rows s, columns t of a pair of tiles: decays times beta (0 above the diagonal)
    auto decays = [&](int t, int s0) __attribute__((always_inline)) {
        f32x4 e;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = gt.decay(t, s0 + i) * gt.beta[s0 + i];
            e[i] = t >= s0 + i ? x : 0.f;
        }
        return e;
    };
    {   // A: columns t of tile w against the rows of every tile up to it
        bf16x8 kt[KB][NT];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) k.get8(16 * w + r, 4 * kb + q, kt[kb]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f32x4 x = {0.f, 0.f, 0.f, 0.f};
            if (j <= w) {
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    bf16x8 ks[NT];
                    k.get8(16 * j + r, 4 * kb + q, ks);
                    x = product<NT, NT>(ks, kt[kb], x);
                }
                x *= decays(16 * w + r, 16 * j + 4 * q);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (j == w && 4 * q + i == r) x[i] = 0.f;  // the diagonal
            }
            *reinterpret_cast<f32x4 *>(&As[16 * w + r][16 * j + 4 * q]) = x;
        }
    }
    // the scores, formed in the orientation in which two tiles are an operand
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
        const int c = w + 4 * m, a = tri_tile(BWD, c), b = tri_block(BWD, c);
        if (c >= 6) continue;
        f32x4 x[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int o = 2 * b + z;  // forward the tile of s, backward of t
            x[z] = (f32x4){0.f, 0.f, 0.f, 0.f};
            if (BWD ? o < a : o > a) continue;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                bf16x8 ks[NT];
                k.get8(16 * (BWD ? a : o) + r, 4 * kb + q, ks);
                x[z] = BWD ? product<NT, NT>(qf[m][BWD ? z : 0][kb], ks, x[z]) : product<NT, NT>(ks, qf[m][0][kb], x[z]);
            }
            if constexpr (BWD) {
                const int s = 16 * a + r;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = 16 * o + 4 * q + i;
                    const float e = gt.decay(t, s) * gt.beta[s];
                    x[z][i] *= t >= s ? e : 0.f;
                }
            } else {
                x[z] *= decays(16 * a + r, 16 * o + 4 * q);
            }
        }
        constexpr int NP = BWD || NT == 3 ? 3 : 2;  // forward, only o reads them
        bf16x8 t[NP];
        split<NP>(x[0], x[1], t);
#pragma unroll
        for (int n = 0; n < NP; ++n) put_fragment(p.pf, head * kDeltaTri + NP * c + n, l, t[n]);
    }
    __syncthreads();
    ut_transform<kUtN + 4>(As, As, Xs, w, l);
    for (int c = w; c < 6; c += 4) {
        const int a = tri_tile(BWD, c), b = tri_block(BWD, c);
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int m = 16 * a + r, n = 32 * b + perm(q, e);
            x[e] = BWD ? As[n][m] : As[m][n];
        }
        bf16x8 t[3];
        split<3>(x, t);
#pragma unroll
        for (int n = 0; n < 3; ++n) put_fragment(p.tf, head * kDeltaTri + 3 * c + n, l, t[n]);
    }
    if (p.raw || hv % p.group) return;  // uniform over the workgroup
    const long key = ((long)slot * p.Hk + hk) * (4 * KB * NT);
#pragma unroll
    for (int m = 0; m < 2; ++m)  // block kb of channels, tile w of tokens, terms
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            bf16x8 t[NT];
            const int row = 16 * w + r, ch = 32 * kb + 8 * q;
            load8<NT>(m ? p.q : p.k, (at.row0 + row) * (m ? p.ldq : p.ldk) + (long)hk * p.dk + ch, row < at.n && ch < p.dk, t);
#pragma unroll
            for (int n = 0; n < NT; ++n) put_fragment(m ? p.qf : p.kf, key + (kb * 4 + w) * NT + n, key_place(r, q), t[n]);
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
    // 16 bytes at a time go only to and from 16-byte places
    const auto aligned = [](const void *x, int64_t ld) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0 && (ld & 7) == 0; };
    p.raw = p.io_bf16 && aligned(p.q, p.ldq) && aligned(p.k, p.ldk);
    p.kf = take(key);  // also where they are not used: the size does not depend on addresses
    p.qf = take(key);
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
