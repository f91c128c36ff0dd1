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

template <int NT, int KB>
struct GradShared {
    union {
        struct {  // a block of 32 columns of the state before, of the gradient behind, of D and of y
            Staged<32 * KB, 3, 32> S, G;
            Staged<64, 3, 32> D, Y;
        };
        struct {  // then the pairs' matrices (rows s, columns t), and q and k (with fp32 one after the other)
            Staged<kDeltaC, NT == 1 ? 2 : 3, kDeltaC> C1, C2;
            Staged<32 * KB, NT, kDeltaC> x[NT == 1 ? 2 : 1];
        };
    };
    float col_m[2][kDeltaC], col_pair[2][kDeltaC], row_m[2][kDeltaC], read[2][kDeltaC], write[2][kDeltaC], dot[4];
    ChunkGates gt;
};

template <int N>
__device__ __forceinline__ float turned(float x) {  // by N lanes within 16
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x120 + N, 0xf, 0xf, true));
}

__device__ __forceinline__ float row_lanes(float x) {  // over the 16 lanes of a quarter
    x += turned<8>(x);
    x += turned<4>(x);
    x += turned<2>(x);
    return x + turned<1>(x);
}

__device__ __forceinline__ float quarters(float x, int l) {  // over the four quarters
    x += of_lane(x, l ^ 16);
    return x + of_lane(x, l ^ 32);
}

// Four waves: wave (th, cq) has token tiles 2 th and 2 th + 1 and half cq of the channels; of pairs of tokens the s
// tiles cq and cq + 2.  Two workgroups fit a compute unit: one waits while the other works (4 x 4,096 tokens, 16 heads of 128 x 128,
// bf16: 326 us at best, 356 on the mean; eight waves and one workgroup 438 to 540).  It moves 1.21 GB, 3.7 TB/s: four fifths of it
// states and their gradients, each read once; the matrix cores are busy for a quarter of its time.
template <int NT, int KB>
__global__ void __launch_bounds__(256, 2) delta_grad_kernel(DeltaParams p) {
    constexpr int NX = NT == 1 ? 2 : 3;  // terms of what only outputs of the io type read
    constexpr int CT = KB;               // channel tiles of a wave
    __shared__ __attribute__((aligned(16))) GradShared<NT, KB> sh;
    const int hk = blockIdx.x % p.Hk, slot = blockIdx.x / p.Hk;
    const Place at = place_of(p, slot);
    if (at.n <= 0) return;  // uniform over the workgroup
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), th = w >> 1, cq = w & 1;
    const int na = delta_row_tiles(p.dk), nj = delta_col_tiles(p.dv), jblocks = (nj + 1) / 2;
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int h = 0; h < p.group; ++h) {
        int l = tid & 63;
        asm volatile("" : "+v"(l));  // addresses are formed for each head: kept over the heads they would take the registers
        const int r = l & 15, q = l >> 4, mine = 64 * w + l;
        // all of k or q as it lies, 8 channels a turn
        auto bring = [&](const void *x, int64_t ld, auto &to) __attribute__((always_inline)) {
            constexpr int kPieces = kDeltaC * 4 * KB / 256;
            bf16x8 t[kPieces][NT];
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int row = (mine + 256 * i) / (4 * KB), m = (mine + 256 * i) % (4 * KB);
                load8<NT>(x, (at.row0 + row) * ld + (long)hk * p.dk + 8 * m, row < at.n && 8 * m < p.dk, t[i]);
            }
#pragma unroll
            for (int i = 0; i < kPieces; ++i) to.put8((mine + 256 * i) / (4 * KB), (mine + 256 * i) % (4 * KB), t[i]);
        };
        const int hv = hk * p.group + h;
        const long vh = (long)slot * p.Hv + hv;
        // wave w brings column tile w & 1 of a block, half of its row tiles: of S and G, and of D and y
        const float *from = p.ckpt + vh * nj * (na + 4) * 256, *back = p.back + vh * nj * (na + 4) * 256;
        const long dout = (long)hv * p.dv;
        f32x4 a[CT], b[CT], d[2], y[2];
        bf16x8 fo[2][NT];
        auto ask = [&](int jb) __attribute__((always_inline)) {
            const int jt = 2 * jb + (w & 1);
            const long tiles = (long)min(jt, nj - 1) * (na + 4) * 256;
            const int there = jt < nj ? 1024 : 0;  // bytes of a tile
            const Buf s = buffer(from + tiles, there * na), g = buffer(back + tiles, there * na);
            const Buf sd = buffer(from + tiles + na * 256, there * 4), gy = buffer(back + tiles + na * 256, there * 4);
            auto tile = [&](Buf x, int n) __attribute__((always_inline)) {
                return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(x, n * 1024 + l * 16, 0, 0));
            };
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                a[c] = tile(s, (w >> 1) * CT + c);
                b[c] = tile(g, (w >> 1) * CT + c);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                d[c] = tile(sd, (w >> 1) * 2 + c);
                y[c] = tile(gy, (w >> 1) * 2 + c);
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {  // do, by rows: its columns in the operands' order
                const int row = 16 * (2 * th + t) + r, j = 32 * jb + 4 * q;
                load44<NT>(p.dout, (at.row0 + row) * p.Hv * p.dv + dout + j, row < at.n && j < p.dv, row < at.n && j + 16 < p.dv, fo[t]);
            }
        };
        float dot = 0.f;
        if (w == 0) make_gates(p, at, hv, l, sh.gt);
        f32x4 oS[CT][2], yS[CT][2], dG[CT][2], n1[2][2], n2[2][2];  // [channel tile][token tile], [s tile][token tile]
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int c = 0; c < CT; ++c) oS[c][t] = yS[c][t] = dG[c][t] = zero;
            n1[0][t] = n1[1][t] = n2[0][t] = n2[1][t] = zero;
        }
#pragma unroll 1
        for (int jb = 0; jb < jblocks; ++jb) {
            // formed again for each block: kept for all tiles they would take the registers of the sums
            uint32_t pS = Staged<32 * KB, 3, 32>::put_place(16 * (w & 1) + r, q), gS = Staged<32 * KB, 3, 32>::get_place(r, q);
            uint32_t pD = Staged<64, 3, 32>::put_place(16 * (w & 1) + r, q), gD = Staged<64, 3, 32>::get_place(r, q);
            asm volatile("" : "+v"(pS), "+v"(gS), "+v"(pD), "+v"(gD));
            ask(jb);
            lds_barrier();  // the block before is no longer read
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                sh.S.put(pS, (w >> 1) * CT + c, a[c]);
                sh.G.put(pS, (w >> 1) * CT + c, b[c]);
#pragma unroll
                for (int i = 0; i < 4; ++i) dot = fmaf(a[c][i], b[c][i], dot);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                sh.D.put(pD, (w >> 1) * 2 + c, d[c]);
                sh.Y.put(pD, (w >> 1) * 2 + c, y[c]);
            }
            lds_barrier();
            bf16x8 fy[2][3], fd[2][3], s[3], g[3];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                sh.Y.get(gD, 2 * th + t, fy[t]);
                sh.D.get(gD, 2 * th + t, fd[t]);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                if (2 * m > 2 * th + 1) continue;  // above the diagonal
                sh.D.get(gD, 2 * m + cq, s);
                products<3, NT, 2>([&](int, int i) { return s[i]; }, [&](int k, int j) { return fo[k][j]; }, [&](int k) -> f32x4 & { return n1[m][k]; });
                products<3, 3, 2>([&](int, int i) { return s[i]; }, [&](int k, int j) { return fy[k][j]; }, [&](int k) -> f32x4 & { return n2[m][k]; });
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                sh.S.get(gS, cq * CT + c, s);
                sh.G.get(gS, cq * CT + c, g);
                products<3, NT, 2>([&](int, int i) { return s[i]; }, [&](int k, int j) { return fo[k][j]; },
                                   [&](int k) -> f32x4 & { return oS[c][k]; });
                products<3, 3, 4>([&](int k, int i) { return k < 2 ? s[i] : g[i]; }, [&](int k, int j) { return k < 2 ? fy[k][j] : fd[k - 2][j]; },
                                  [&](int k) -> f32x4 & { return k < 2 ? yS[c][k] : dG[c][k - 2]; });
                __builtin_amdgcn_sched_barrier(0);  // no operands of later tiles in registers yet
            }
        }
        __syncthreads();
        if constexpr (NT == 1) {
            bring(p.q, p.ldq, sh.x[0]);
            bring(p.k, p.ldk, sh.x[1]);
        }
        // tile t of the rows of k or q, block kb of channels
        auto rows = [&](bool key, int t, int kb, bf16x8 (&to)[NT]) __attribute__((always_inline)) {
            if constexpr (NT == 1) {
                sh.x[key].get8(16 * t + r, 4 * kb + q, to);
            } else {
                const int row = 16 * t + r, c = 32 * kb + 8 * q;
                load8<NT>(key ? p.k : p.q, (at.row0 + row) * (key ? p.ldk : p.ldq) + (long)hk * p.dk + c, row < at.n && c < p.dk, to);
            }
        };
        __syncthreads();
        // pairs of tokens: rows s of tiles cq and cq + 2, columns t
        float rm[2] = {0.f, 0.f};
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int sa = 2 * m + cq, s0 = 16 * sa + 4 * q;
            float cm[4] = {}, cp[4] = {};
            const f32x4 betas = *reinterpret_cast<const f32x4 *>(&sh.gt.beta[s0]);
            double Ps[4];
            int cuts[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                Ps[i] = sh.gt.P[s0 + i];
                cuts[i] = sh.gt.cut[s0 + i];
            }
            bf16x8 s[KB][NT];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) rows(true, sa, kb, s[kb]);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int ta = 2 * th + t, tt = 16 * ta + r;
                f32x4 c1 = zero, c2 = zero;
                if (sa <= ta) {
                    f32x4 qk = zero, kk = zero;
                    const double Pt = sh.gt.P[tt];
                    const int cut = sh.gt.cut[tt];
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb) {
                        bf16x8 tq[NT], tk[NT];
                        rows(false, ta, kb, tq);
                        rows(true, ta, kb, tk);
                        products<NT, NT, 2>([&](int, int i) { return s[kb][i]; }, [&](int k, int j) { return k ? tk[j] : tq[j]; },
                                            [&](int k) -> f32x4 & { return k ? kk : qk; });
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int s = s0 + i;
                        const float x = sh.gt.power((float)(Pt - Ps[i])), e = tt >= s && cut == cuts[i] ? x : 0.f;
                        const float a1 = tt >= s ? n1[m][t][i] : 0.f, a2 = tt > s ? n2[m][t][i] : 0.f;
                        c1[i] = e * betas[i] * a1;
                        c2[i] = -e * betas[i] * a2;
                        const float pair = tt >= s ? e * (a1 * qk[i] - a2 * kk[i]) : 0.f;
                        cp[i] += pair;
                        const float through = tt > s ? pair * betas[i] : 0.f;  // a token's own pair does not pass its gate
                        rm[t] += through;
                        cm[i] += through;
                    }
                }
                sh.C1.put(sh.C1.put_place(tt, q), sa, c1);
                sh.C2.put(sh.C2.put_place(tt, q), sa, c2);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = row_lanes(cm[i]), z = row_lanes(cp[i]);
                if (r == 0) {
                    sh.col_m[th][s0 + i] = x;
                    sh.col_pair[th][s0 + i] = z;
                }
            }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            rm[t] = quarters(rm[t], l);
            if (q == 0) sh.row_m[cq][16 * (2 * th + t) + r] = rm[t];
        }
        // what the states give, and its dot products with q and k
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int ta = 2 * th + t, tt = 16 * ta + r;
            const float front = sh.gt.front[tt], behind = sh.gt.behind[tt], beta = sh.gt.beta[tt];
            float read = 0.f, write = 0.f;
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                bf16x8 tq[NT], tk[NT];
                rows(false, ta, (cq * CT + c) / 2, tq);
                rows(true, ta, (cq * CT + c) / 2, tk);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float qv = 0.f, kv = 0.f;
#pragma unroll
                    for (int n = NT - 1; n >= 0; --n) {  // an even tile has the first four of the lane's eight channels
                        const uint32_t x = __builtin_bit_cast(u32x4, tq[n])[c % 2 * 2 + i / 2], z = __builtin_bit_cast(u32x4, tk[n])[c % 2 * 2 + i / 2];
                        qv += __uint_as_float(i & 1 ? x & 0xffff0000u : x << 16);
                        kv += __uint_as_float(i & 1 ? z & 0xffff0000u : z << 16);
                    }
                    const float fo_ = front * oS[c][t][i], fy_ = front * yS[c][t][i], bg = behind * dG[c][t][i];
                    oS[c][t][i] = fo_;
                    dG[c][t][i] = fmaf(beta, bg, -fy_);
                    read += qv * fo_ - kv * fy_;
                    write = fmaf(kv, bg, write);
                }
            }
            read = quarters(read, l);
            write = quarters(write, l);
            if (q == 0) {
                sh.read[cq][tt] = read;
                sh.write[cq][tt] = write;
            }
        }
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) dot += of_lane(dot, l ^ s);
        if (l == 0) sh.dot[w] = dot;
        __syncthreads();
        if (w == 0) {
            float db = 0.f, down = 0.f, dots = 0.f;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                db += sh.write[m][l];
                down += sh.read[m][l] + sh.row_m[m][l];
            }
            float up = db * sh.gt.beta[l];
            const float mine = up;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                db += sh.col_pair[m][l];
                down -= sh.col_m[m][l];
            }
#pragma unroll
            for (int s = 1; s < 64; s <<= 1) {  // sums over this token and the later ones, and over the earlier ones
                const float x = of_lane(down, l + s), z = of_lane(up, l - s);
                if (l + s < 64) down += x;
                if (l >= s) up += z;
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) dots += sh.dot[m];
            const float kept = sh.gt.whole * dots;
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
            if constexpr (NT == 3) {
                if (side) __syncthreads();
                bring(side ? p.k : p.q, side ? p.ldk : p.ldq, sh.x[0]);
                __syncthreads();
            }
            const uint32_t gx = Staged<32 * KB, NT, kDeltaC>::key_get_place(r, q), gc = sh.C1.get_place(r, q);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                bf16x8 c1[2][NX], c2[2][NX], c2t[2][NX];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int ta = 2 * th + t;
                    const uint32_t pc = sh.C1.put_place(16 * ta + r, q);
                    if (side) {
                        sh.C1.column(pc, b, c1[t]);
                        sh.C2.column(pc, b, c2[t]);
                        sh.C2.get(gc, ta, c2t[t], b);
                    } else {
                        sh.C1.get(gc, ta, c1[t], b);
                    }
                }
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    bf16x8 xt[NT];
                    sh.x[NT == 1 ? side : 0].key_get(gx, cq * CT + c, b, xt);
                    if (side) {
                        products<NT, NX, 4>([&](int, int i) { return xt[i]; }, [&](int k, int j) { return k < 2 ? c1[k][j] : c2[k - 2][j]; },
                                            [&](int k) -> f32x4 & { return k < 2 ? oS[c][k] : dG[c][k - 2]; });
                        products<NT, NX, 2>([&](int, int i) { return xt[i]; }, [&](int k, int j) { return c2t[k][j]; },
                                            [&](int k) -> f32x4 & { return dG[c][k]; });
                    } else {
                        products<NT, NX, 2>([&](int, int i) { return xt[i]; }, [&](int k, int j) { return c1[k][j]; },
                                            [&](int k) -> f32x4 & { return dG[c][k]; });
                    }
                }
            }
        }
        // a shared key head's gradients are summed over its value heads, always in the same order
        const bool last = h == p.group - 1;
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (p.group > 1) {
                    f32x4 *sum = reinterpret_cast<f32x4 *>(p.sum) + ((((long)slot * p.Hk + hk) * 4 + w) * CT + c) * 256 + t * 128 + l;
                    if (h) {
                        oS[c][t] += sum[0];
                        dG[c][t] += sum[64];
                    }
                    if (!last) {
                        sum[0] = oS[c][t];
                        sum[64] = dG[c][t];
                    }
                }
                const int row = 16 * (2 * th + t) + r, tile = cq * CT + c, chan = 32 * (tile / 2) + 8 * q + 4 * (tile % 2);
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
        if (!last) __syncthreads();
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
