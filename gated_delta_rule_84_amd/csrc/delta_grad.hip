// delta_grad.hip -- the gradients of q, k and the gates of the delta rule, chunk by chunk (delta.hpp).
//
// With S the state before the chunk, G the gradient of the state behind it, D and y of its tokens,
//     N1 = do D^T, N2 = y D^T,   C1 = e beta (.) N1 (t >= s),   C2 = -e beta (.) N2 (t > s)
//     dq = front (do S^T) + C1 k
//     dk = C1^T q + (C2 + C2^T) k - front (y S^T) + behind beta (D G^T)
//     dbeta_s = sum_t e_ts (N1 q.k - N2 k.k)_ts + behind_s k_s.(D G^T)_s
// and the gradient of a log gate is the sum of what passes it: from the state before to the one behind,
// from earlier writes to the state behind, from the state before to later reads, from earlier writes to
// later reads.
//
// Products are formed with channels as rows and tokens as columns, so that a lane's results are four
// channels of one token: q and k of the dot products lie in its fragments already, gates are one value a lane,
// and stores are whole words.  All contractions over the value's columns run in one pass over
// blocks of 32 of them, which are split into terms once, into shared memory, column by column; the
// transposing LDS read turns them into operands.
#include "delta.hpp"

namespace gdr {
namespace {

constexpr int kLC = kDeltaC + 4;

template <int NT, int KB>
struct GradShared {
    union {
        struct {
            Staged<32 * KB, 3, 32> S, G;
            Staged<64, 3, 32> D, Y;
        };
        struct {
            float C1[kDeltaC][kLC], C2[kDeltaC][kLC];  // [t][s]
            Staged<32 * KB, NT, kDeltaC> x;            // k or q
        };
    };
    float col_m[2][kDeltaC], col_pair[2][kDeltaC], row_m[2][kDeltaC], read[2][kDeltaC], write[2][kDeltaC], dot[4];
    ChunkGates gt;
};

__device__ __forceinline__ float row_lanes(float x) {  // over the 16 lanes of a quarter
#pragma unroll
    for (int s = 1; s < 16; s <<= 1) x += __shfl_xor(x, s);
    return x;
}

__device__ __forceinline__ float quarters(float x) {  // over the four quarters
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// Four waves: wave (th, ch) has token tiles 2 th and 2 th + 1 and half ch of the channels.
template <int NT, int KB>
__global__ void __launch_bounds__(256, 2) delta_grad_kernel(DeltaParams p) {
    constexpr int NX = NT == 1 ? 2 : 3;  // terms of what only outputs of the io type read
    __shared__ __attribute__((aligned(16))) GradShared<NT, KB> sh;
    const int hk = blockIdx.x % p.Hk, slot = blockIdx.x / p.Hk;
    const Place at = place_of(p, slot);
    if (at.n <= 0) return;  // uniform over the workgroup
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), th = w >> 1, ch = w & 1;
    const int na = delta_row_tiles(p.dk), nj = delta_col_tiles(p.dv), jblocks = (nj + 1) / 2;
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int h = 0; h < p.group; ++h) {
        int l = tid & 63;
        asm volatile("" : "+v"(l));  // addresses are formed for each head: kept over the heads they would take the registers
        const int r = l & 15, q = l >> 4;
        const int hv = hk * p.group + h;
        const long vh = (long)slot * p.Hv + hv, base = vh * nj * (na + 4) * 256;
        const float *ST = p.ckpt + base, *GT = p.back + base;
        if (h) __syncthreads();
        if (w == 0) make_gates(p, at, hv, l, sh.gt);
        f32x4 oS[KB][2], yS[KB][2], dG[KB][2], n1[2][2], n2[2][2];  // [channel tile][token tile], [s tile][token tile]
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int c = 0; c < KB; ++c) oS[c][t] = yS[c][t] = dG[c][t] = zero;
            n1[0][t] = n1[1][t] = n2[0][t] = n2[1][t] = zero;
        }
        float dot = 0.f;
#pragma unroll 1
        for (int jb = 0; jb < jblocks; ++jb) {
            // formed again for each block: kept for all tiles they would take the registers of the sums
            uint32_t pS = Staged<32 * KB, 3, 32>::put_place(16 * (w & 1) + r, q), gS = Staged<32 * KB, 3, 32>::get_place(r, q);
            uint32_t pD = Staged<64, 3, 32>::put_place(16 * (w & 1) + r, q), gD = Staged<64, 3, 32>::get_place(r, q);
            asm volatile("" : "+v"(pS), "+v"(gS), "+v"(pD), "+v"(gD));
            // wave w brings column tile w & 1 of the block, half of its row tiles
            {
                const int jt = 2 * jb + (w & 1);
                const bool there = jt < nj;
                const float *s = ST + (long)jt * (na + 4) * 256 + l * 4, *g = GT + (long)jt * (na + 4) * 256 + l * 4;
                f32x4 a[KB], b[KB], d[2], y[2];
#pragma unroll
                for (int c = 0; c < KB; ++c) {
                    const int tile = (w >> 1) * KB + c;
                    a[c] = b[c] = zero;
                    if (there && tile < na) {
                        a[c] = *reinterpret_cast<const f32x4 *>(s + tile * 256);
                        b[c] = *reinterpret_cast<const f32x4 *>(g + tile * 256);
                    }
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int tile = na + (w >> 1) * 2 + c;
                    d[c] = y[c] = zero;
                    if (there) {
                        d[c] = *reinterpret_cast<const f32x4 *>(s + tile * 256);
                        y[c] = *reinterpret_cast<const f32x4 *>(g + tile * 256);
                    }
                }
                __syncthreads();  // the block before is no longer read
#pragma unroll
                for (int c = 0; c < KB; ++c) {
                    sh.S.put(pS, (w >> 1) * KB + c, a[c]);
                    sh.G.put(pS, (w >> 1) * KB + c, b[c]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) dot = fmaf(a[c][i], b[c][i], dot);
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    sh.D.put(pD, (w >> 1) * 2 + c, d[c]);
                    sh.Y.put(pD, (w >> 1) * 2 + c, y[c]);
                }
            }
            bf16x8 fo[2][NT], fy[2][3], fd[2][3];
#pragma unroll
            for (int t = 0; t < 2; ++t) {  // do, by rows: its columns in the operands' order
                const int row = 16 * (2 * th + t) + r;
                const long o = ((at.row0 + row) * p.Hv + hv) * p.dv;
                const int j = 32 * jb + 4 * q;
                load44<NT>(p.dout, o + j, row < at.n && j < p.dv, row < at.n && j + 16 < p.dv, fo[t]);
            }
            __syncthreads();
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                sh.Y.get(gD, 2 * th + t, fy[t]);
                sh.D.get(gD, 2 * th + t, fd[t]);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int sa = 2 * m + ch;  // s tiles of this wave
                if (sa > 2 * th + 1) continue;
                bf16x8 d[3];
                sh.D.get(gD, sa, d);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (sa > 2 * th + t) continue;
                    n1[m][t] = product<3, NT>(d, fo[t], n1[m][t]);
                    n2[m][t] = product<3, 3>(d, fy[t], n2[m][t]);
                }
            }
#pragma unroll
            for (int c = 0; c < KB; ++c) {
                bf16x8 s[3], g[3];
                sh.S.get(gS, ch * KB + c, s);
                sh.G.get(gS, ch * KB + c, g);
                products<3, NT, 2>([&](int, int i) { return s[i]; }, [&](int k, int j) { return fo[k][j]; },
                                   [&](int k) -> f32x4 & { return oS[c][k]; });
                products<3, 3, 4>([&](int k, int i) { return k < 2 ? s[i] : g[i]; }, [&](int k, int j) { return k < 2 ? fy[k][j] : fd[k - 2][j]; },
                                  [&](int k) -> f32x4 & { return k < 2 ? yS[c][k] : dG[c][k - 2]; });
                __builtin_amdgcn_sched_barrier(0);  // no operands of later tiles in registers yet
            }
        }
        // tile t of the rows of k or q, block kb of channels
        auto rows = [&](const void *x, int64_t ld, int t, int kb, bf16x8 (&to)[NT]) __attribute__((always_inline)) {
            const int row = 16 * t + r, c = 32 * kb + 8 * q;
            load8<NT>(x, (at.row0 + row) * ld + (long)hk * p.dk + c, row < at.n && c < p.dk, to);
        };
        __syncthreads();
        // pairs of tokens: rows s, columns t
        float cm[2][4] = {}, cp[2][4] = {}, rm[2] = {0.f, 0.f};
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int ta = 2 * th + t, tt = 16 * ta + r;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int sa = 2 * m + ch;
                f32x4 c1 = zero, c2 = zero;
                __builtin_amdgcn_sched_barrier(0);
                if (sa <= ta) {
                    f32x4 qk = zero, kk = zero;
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb) {
                        bf16x8 s[NT], tq[NT], tk[NT];
                        rows(p.k, p.ldk, sa, kb, s);
                        rows(p.q, p.ldq, ta, kb, tq);
                        rows(p.k, p.ldk, ta, kb, tk);
                        qk = product<NT, NT>(s, tq, qk);
                        kk = product<NT, NT>(s, tk, kk);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int s = 16 * sa + 4 * q + i;
                        const float e = tt >= s ? sh.gt.decay(tt, s) : 0.f, beta = sh.gt.beta[s];
                        const float a1 = tt >= s ? n1[m][t][i] : 0.f, a2 = tt > s ? n2[m][t][i] : 0.f;
                        c1[i] = e * beta * a1;
                        c2[i] = -e * beta * a2;
                        const float pair = tt >= s ? e * (a1 * qk[i] - a2 * kk[i]) : 0.f;
                        cp[m][i] += pair;
                        if (tt > s) {  // a token's own pair does not pass its gate
                            rm[t] += pair * beta;
                            cm[m][i] += pair * beta;
                        }
                    }
                }
                *reinterpret_cast<f32x4 *>(&sh.C1[tt][16 * sa + 4 * q]) = c1;
                *reinterpret_cast<f32x4 *>(&sh.C2[tt][16 * sa + 4 * q]) = c2;
            }
            rm[t] = quarters(rm[t]);
            if (q == 0) sh.row_m[ch][tt] = rm[t];
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = row_lanes(cm[m][i]), z = row_lanes(cp[m][i]);
                if (r == 0) {
                    sh.col_m[th][16 * (2 * m + ch) + 4 * q + i] = x;
                    sh.col_pair[th][16 * (2 * m + ch) + 4 * q + i] = z;
                }
            }
        // what the states give, and its dot products with q and k
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int ta = 2 * th + t, tt = 16 * ta + r;
            const float front = sh.gt.front[tt], behind = sh.gt.behind[tt], beta = sh.gt.beta[tt];
            float read = 0.f, write = 0.f;
#pragma unroll
            for (int c = 0; c < KB; c += 2) {
                const int kb = (ch * KB + c) / 2;
                __builtin_amdgcn_sched_barrier(0);
                float qv[8], kv[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) qv[e] = kv[e] = 0.f;
                bf16x8 tq[NT], tk[NT];
                rows(p.q, p.ldq, ta, kb, tq);
                rows(p.k, p.ldk, ta, kb, tk);
#pragma unroll
                for (int n = NT - 1; n >= 0; --n) {
                    const u32x4 a = __builtin_bit_cast(u32x4, tq[n]), b = __builtin_bit_cast(u32x4, tk[n]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        qv[e] += __uint_as_float(e & 1 ? a[e / 2] & 0xffff0000u : a[e / 2] << 16);
                        kv[e] += __uint_as_float(e & 1 ? b[e / 2] & 0xffff0000u : b[e / 2] << 16);
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int cc = c + e / 4, i = e % 4;
                    const float fo = front * oS[cc][t][i], fy = front * yS[cc][t][i], bg = behind * dG[cc][t][i];
                    oS[cc][t][i] = fo;
                    dG[cc][t][i] = fmaf(beta, bg, -fy);
                    read += qv[e] * fo - kv[e] * fy;
                    write = fmaf(kv[e], bg, write);
                }
            }
            read = quarters(read);
            write = quarters(write);
            if (q == 0) {
                sh.read[ch][tt] = read;
                sh.write[ch][tt] = write;
            }
        }
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) dot += __shfl_xor(dot, s);
        if (l == 0) sh.dot[w] = dot;
        __syncthreads();
        if (w == 0) {
            float db = sh.write[0][l] + sh.write[1][l], up = db * sh.gt.beta[l];
            float down = sh.read[0][l] + sh.read[1][l] + sh.row_m[0][l] + sh.row_m[1][l];
            const float mine = up;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                db += sh.col_pair[m][l];
                down -= sh.col_m[m][l];
            }
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {  // sums over this token and the later ones, and over the earlier ones
                const float x = __shfl_down(down, d), y = __shfl_up(up, d);
                if (l + d < 64) down += x;
                if (l >= d) up += y;
            }
            const float kept = sh.gt.whole * (sh.dot[0] + sh.dot[1] + sh.dot[2] + sh.dot[3]);
            const bool cuts = l ? sh.gt.cut[l] != sh.gt.cut[l - 1] : sh.gt.cut[0] != 0;
            if (l < at.n) {
                const long o = (at.row0 + l) * p.Hv + hv;
                st_elem(p.dg, o, cuts ? 0.f : kept + (up - mine) + down, p.gate_bf16);
                st_elem(p.db, o, db, p.gate_bf16);
            }
        }
        // + C1^T q to dk, + C1 k to dq and (C2 + C2^T) k to dk
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            if (side) __syncthreads();
            constexpr int kPieces = kDeltaC * 4 * KB / 256;
            bf16x8 x[kPieces][NT];
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int row = (tid + 256 * i) / (4 * KB), m = (tid + 256 * i) % (4 * KB);
                load8<NT>(side ? p.k : p.q, (at.row0 + row) * (side ? p.ldk : p.ldq) + (long)hk * p.dk + 8 * m, row < at.n && 8 * m < p.dk, x[i]);
            }
#pragma unroll
            for (int i = 0; i < kPieces; ++i) sh.x.put8((tid + 256 * i) / (4 * KB), (tid + 256 * i) % (4 * KB), x[i]);
            __syncthreads();
            const uint32_t gx = Staged<32 * KB, NT, kDeltaC>::key_get_place(r, q);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                bf16x8 c1[2][NX], c2[2][NX];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    float x1[8], x2[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int m = 16 * (2 * th + t) + r, o = 32 * b + perm(q, e);
                        x1[e] = side ? sh.C1[m][o] : sh.C1[o][m];
                        if (side) x2[e] = sh.C2[m][o] + sh.C2[o][m];
                    }
                    split<NX>(x1, c1[t]);
                    if (side) split<NX>(x2, c2[t]);
                }
#pragma unroll
                for (int c = 0; c < KB; ++c) {
                    bf16x8 xt[NT];
                    sh.x.key_get(gx, ch * KB + c, b, xt);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (side) {
                            oS[c][t] = product<NT, NX>(xt, c1[t], oS[c][t]);
                            dG[c][t] = product<NT, NX>(xt, c2[t], dG[c][t]);
                        } else {
                            dG[c][t] = product<NT, NX>(xt, c1[t], dG[c][t]);
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        // a shared key head's gradients are summed over its value heads, always in the same order
        const bool last = h == p.group - 1;
#pragma unroll
        for (int c = 0; c < KB; ++c)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (p.group > 1) {
                    f32x4 *sum = reinterpret_cast<f32x4 *>(p.sum) + ((((long)slot * p.Hk + hk) * 4 + w) * KB + c) * 256 + t * 128 + l;
                    if (h) {
                        oS[c][t] += sum[0];
                        dG[c][t] += sum[64];
                    }
                    if (!last) {
                        sum[0] = oS[c][t];
                        sum[64] = dG[c][t];
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                const int row = 16 * (2 * th + t) + r, tile = ch * KB + c, chan = 32 * (tile / 2) + 8 * q + 4 * (tile % 2);
                if (!last || row >= at.n || chan >= p.dk) continue;
                const long o = ((at.row0 + row) * p.Hk + hk) * p.dk + chan;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const f32x4 x = m ? dG[c][t] : oS[c][t];
                    void *out = m ? p.dkk : p.dq;
                    if constexpr (NT == 1) {
                        typedef uint32_t wu2 __attribute__((ext_vector_type(2), aligned(2)));
                        *reinterpret_cast<wu2 *>(static_cast<uint16_t *>(out) + o) = (wu2){pk_bf16(x[0], x[1]), pk_bf16(x[2], x[3])};
                    } else {
                        typedef float wf4 __attribute__((ext_vector_type(4), aligned(4)));
                        *reinterpret_cast<wf4 *>(static_cast<float *>(out) + o) = (wf4){x[0], x[1], x[2], x[3]};
                    }
                }
            }
    }
}

}  // namespace

hipError_t launch_delta_grad(const DeltaParams &p0, hipStream_t s) {
    DeltaParams p = p0;
    void *args[] = {&p};
    const int kb = delta_blocks(p.dk);
    const void *fn = p.io_bf16 ? (kb == 2 ? reinterpret_cast<const void *>(&delta_grad_kernel<1, 2>) : reinterpret_cast<const void *>(&delta_grad_kernel<1, 4>))
                               : (kb == 2 ? reinterpret_cast<const void *>(&delta_grad_kernel<3, 2>) : reinterpret_cast<const void *>(&delta_grad_kernel<3, 4>));
    return hipLaunchKernel(fn, dim3((unsigned)p.nslot * p.Hk), dim3(256), args, 0, s);
}

}  // namespace gdr
