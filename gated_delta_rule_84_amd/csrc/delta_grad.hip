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
#include "delta.hpp"

namespace gdr {
namespace {

constexpr int kLC = kDeltaC + 4;

template <int JB>
struct GradShared {
    static constexpr int LJ = 32 * JB + 8;
    union {
        uint16_t D[3][kDeltaC][LJ];
        uint16_t SG[2][3][32][LJ];
    };
    union {
        struct {
            float C1[kDeltaC][kLC], C2[kDeltaC][kLC];
        };
        float qk[2][kDeltaC][36];  // q and k of 32 channels
    };
    float col_m[4][kDeltaC], col_pair[4][kDeltaC], row_m[2][kDeltaC], read[2][kDeltaC], write[2][kDeltaC], dot[8];
    ChunkGates gt;
};

__device__ __forceinline__ float row_lanes(float x) {  // over the 16 lanes of a row of tiles
#pragma unroll
    for (int s = 1; s < 16; s <<= 1) x += __shfl_xor(x, s);
    return x;
}

__device__ __forceinline__ float column_lanes(float x) {  // over the four quarters
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// Eight waves: w has the 16-row tile w of tokens; of each 32 channels half hf's 16.
template <int NT, int KB, int JB>
__global__ void __launch_bounds__(512) delta_grad_kernel(DeltaParams p) {
    constexpr int NX = NT == 1 ? 2 : 3;  // terms of what only outputs of the io type read
    __shared__ __attribute__((aligned(16))) GradShared<JB> sh;
    const int hk = blockIdx.x % p.Hk, slot = blockIdx.x / p.Hk;
    const Place at = place_of(p, slot);
    if (at.n <= 0) return;  // uniform over the workgroup
    const int tid = threadIdx.x, w = tid >> 6 & 3, hf = tid >> 8, l = tid & 63, r = l & 15, q = l >> 4;
    const long key = ((long)slot * p.Hk + hk) * (4 * KB * NT);
    const long sstate = (long)p.dk * p.dv, sckpt = sstate + (long)kDeltaC * p.dv;
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    f32x4 dq[KB], dk[KB];
#pragma unroll
    for (int a = 0; a < KB; ++a) dq[a] = dk[a] = zero;
    const int trow = 16 * w + 4 * q;  // first of the lane's rows
    for (int h = 0; h < p.group; ++h) {
        const int hv = hk * p.group + h;
        const long vh = (long)slot * p.Hv + hv;
        const float *S = p.ckpt + vh * sckpt, *D = S + sstate, *G = p.G + vh * sstate, *Y = p.y + vh * ((long)kDeltaC * p.dv);
        if (h) __syncthreads();
        if (tid < 64) make_gates(p, at, hv, l, sh.gt);
        bf16x8 dof[JB][NT], yf[JB][3], df[JB][3];
#pragma unroll
        for (int jb = 0; jb < JB; ++jb) {
            const int j = 32 * jb + 8 * q, t = 16 * w + r;
            load8<NT>(p.dout, ((at.row0 + t) * p.Hv + hv) * p.dv + j, t < at.n && j < p.dv, dof[jb]);
            load8<3>(Y, (long)t * p.dv + j, j < p.dv, yf[jb]);
        }
        for (int i = tid; i < kDeltaC * 4 * JB; i += 512) {
            const int t = i / (4 * JB), j = i % (4 * JB) * 8;
            bf16x8 x[3];
            load8<3>(D, (long)t * p.dv + j, j < p.dv, x);
#pragma unroll
            for (int n = 0; n < 3; ++n) *reinterpret_cast<bf16x8 *>(&sh.D[n][t][j]) = x[n];
        }
        __syncthreads();
#pragma unroll
        for (int jb = 0; jb < JB; ++jb)
#pragma unroll
            for (int n = 0; n < 3; ++n) df[jb][n] = *reinterpret_cast<const bf16x8 *>(&sh.D[n][16 * w + r][32 * jb + 8 * q]);
        float rm[4] = {0.f, 0.f, 0.f, 0.f};
        for (int j = hf; j < 4; j += 2) {
            f32x4 n1 = zero, n2 = zero, qk = zero, kk = zero;
            if (j <= w) {
#pragma unroll
                for (int jb = 0; jb < JB; ++jb) {
                    bf16x8 b[3];
#pragma unroll
                    for (int n = 0; n < 3; ++n) b[n] = *reinterpret_cast<const bf16x8 *>(&sh.D[n][16 * j + r][32 * jb + 8 * q]);
                    n1 = product<NT, 3>(dof[jb], b, n1);
                    n2 = product<3, 3>(yf[jb], b, n2);
                }
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    bf16x8 b[NT], aq[NT], ak[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        b[n] = fragment(p.kf, key + (j * KB + kb) * NT + n, l);
                        aq[n] = fragment(p.qf, key + (w * KB + kb) * NT + n, l);
                        ak[n] = fragment(p.kf, key + (w * KB + kb) * NT + n, l);
                    }
                    qk = product<NT, NT>(aq, b, qk);
                    kk = product<NT, NT>(ak, b, kk);
                }
            }
            const int s = 16 * j + r;
            const float beta = sh.gt.beta[s];
            float cm = 0.f, cp = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = trow + i;
                const float e = t >= s ? sh.gt.decay(t, s) : 0.f;
                const float a1 = t >= s ? n1[i] : 0.f, a2 = t > s ? n2[i] : 0.f;
                sh.C1[t][s] = e * beta * a1;
                sh.C2[t][s] = -e * beta * a2;
                const float pair = t >= s ? e * (a1 * qk[i] - a2 * kk[i]) : 0.f;
                cp += pair;
                if (t > s) {  // a token's own pair does not pass its gate
                    rm[i] += pair * beta;
                    cm += pair * beta;
                }
            }
            cm = column_lanes(cm);
            cp = column_lanes(cp);
            if (q == 0) {
                sh.col_m[w][s] = cm;
                sh.col_pair[w][s] = cp;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = row_lanes(rm[i]);
            if (r == 0) sh.row_m[hf][trow + i] = x;
        }
        __syncthreads();
        // C1 k, C1^T q, (C2 + C2^T) k
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            float x1[8], x1t[8], x2[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int m = 16 * w + r, o = 32 * b + perm(q, e);
                x1[e] = sh.C1[m][o];
                x1t[e] = sh.C1[o][m];
                x2[e] = sh.C2[m][o] + sh.C2[o][m];
            }
            bf16x8 c1[NX], c1t[NX], c2[NX];
            split<NX>(x1, c1);
            split<NX>(x1t, c1t);
            split<NX>(x2, c2);
#pragma unroll
            for (int a = 0; a < KB; ++a) {
                bf16x8 kt[NT], qt[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    kt[n] = fragment(p.ktf, key + ((2 * a + hf) * 2 + b) * NT + n, l);
                    qt[n] = fragment(p.qtf, key + ((2 * a + hf) * 2 + b) * NT + n, l);
                }
                dq[a] = product<NX, NT>(c1, kt, dq[a]);
                dk[a] = product<NX, NT>(c1t, qt, dk[a]);
                dk[a] = product<NX, NT>(c2, kt, dk[a]);
            }
        }
        float read[4] = {0.f, 0.f, 0.f, 0.f}, write[4] = {0.f, 0.f, 0.f, 0.f}, dot = 0.f;
#pragma unroll
        for (int cb = 0; cb < KB; ++cb) {
            __syncthreads();  // the last reads of D or of the block before
            {
                const int m = tid >> 8, t = tid >> 2 & 63, c = (tid & 3) * 8, ch = 32 * cb + c;
                const void *from = m ? p.k : p.q;
                const long o = (at.row0 + t) * (m ? p.ldk : p.ldq) + (long)hk * p.dk + ch;
                const bool there = t < at.n && ch < p.dk;
#pragma unroll
                for (int e = 0; e < 8; ++e) sh.qk[m][t][c + e] = there ? ld_elem(from, o + e, NT == 1) : 0.f;
            }
            for (int i = tid; i < 32 * 4 * JB; i += 512) {
                const int c = i / (4 * JB), j = i % (4 * JB) * 8, ch = 32 * cb + c;
                const bool there = ch < p.dk && j < p.dv;
                float x[2][8];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const float *from = (m ? G : S) + (long)ch * p.dv + j;
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        f32x4 z = zero;
                        if (there) z = *reinterpret_cast<const f32x4 *>(from + e);
#pragma unroll
                        for (int i4 = 0; i4 < 4; ++i4) x[m][e + i4] = z[i4];
                    }
                    bf16x8 t[3];
                    split<3>(x[m], t);
#pragma unroll
                    for (int n = 0; n < 3; ++n) *reinterpret_cast<bf16x8 *>(&sh.SG[m][n][c][j]) = t[n];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) dot = fmaf(x[0][e], x[1][e], dot);
            }
            __syncthreads();
            f32x4 oS = zero, yS = zero, dG = zero;
#pragma unroll
            for (int jb = 0; jb < JB; ++jb) {
                bf16x8 s[3], g[3];
#pragma unroll
                for (int n = 0; n < 3; ++n) {
                    s[n] = *reinterpret_cast<const bf16x8 *>(&sh.SG[0][n][16 * hf + r][32 * jb + 8 * q]);
                    g[n] = *reinterpret_cast<const bf16x8 *>(&sh.SG[1][n][16 * hf + r][32 * jb + 8 * q]);
                }
                oS = product<NT, 3>(dof[jb], s, oS);
                yS = product<3, 3>(yf[jb], s, yS);
                dG = product<3, 3>(df[jb], g, dG);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = trow + i;
                const float qv = sh.qk[0][t][16 * hf + r], kv = sh.qk[1][t][16 * hf + r];
                const float fo = sh.gt.front[t] * oS[i], fy = sh.gt.front[t] * yS[i], bg = sh.gt.behind[t] * dG[i];
                dq[cb][i] += fo;
                dk[cb][i] += fmaf(sh.gt.beta[t], bg, -fy);
                read[i] += qv * fo - kv * fy;
                write[i] = fmaf(kv, bg, write[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = row_lanes(read[i]), z = row_lanes(write[i]);
            if (r == 0) {
                sh.read[hf][trow + i] = x;
                sh.write[hf][trow + i] = z;
            }
        }
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) dot += __shfl_xor(dot, s);
        if (l == 0) sh.dot[tid >> 6] = dot;
        __syncthreads();
        if (tid < 64) {
            float db = sh.write[0][l] + sh.write[1][l], up = db * sh.gt.beta[l];
            float down = sh.read[0][l] + sh.read[1][l] + sh.row_m[0][l] + sh.row_m[1][l], dots = 0.f;
            const float mine = up;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                db += sh.col_pair[m][l];
                down -= sh.col_m[m][l];
            }
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {  // sums over this token and the later ones, and over the earlier ones
                const float x = __shfl_down(down, d), y = __shfl_up(up, d);
                if (l + d < 64) down += x;
                if (l >= d) up += y;
            }
#pragma unroll
            for (int m = 0; m < 8; ++m) dots += sh.dot[m];
            const float kept = sh.gt.whole * dots;
            const bool cuts = l ? sh.gt.cut[l] != sh.gt.cut[l - 1] : sh.gt.cut[0] != 0;
            if (l < at.n) {
                const long o = (at.row0 + l) * p.Hv + hv;
                st_elem(p.dg, o, cuts ? 0.f : kept + (up - mine) + down, p.gate_bf16);
                st_elem(p.db, o, db, p.gate_bf16);
            }
        }
    }
#pragma unroll
    for (int a = 0; a < KB; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = trow + i, ch = 32 * a + 16 * hf + r;
            if (t >= at.n || ch >= p.dk) continue;
            const long o = ((at.row0 + t) * p.Hk + hk) * p.dk + ch;
            st_elem(p.dq, o, dq[a][i], NT == 1);
            st_elem(p.dkk, o, dk[a][i], NT == 1);
        }
}

template <int NT, int KB>
const void *pick(int jb) {
    return jb == 2 ? reinterpret_cast<const void *>(&delta_grad_kernel<NT, KB, 2>) : reinterpret_cast<const void *>(&delta_grad_kernel<NT, KB, 4>);
}

}  // namespace

hipError_t launch_delta_grad(const DeltaParams &p0, hipStream_t s) {
    DeltaParams p = p0;
    void *args[] = {&p};
    const int kb = delta_blocks(p.dk), jb = delta_blocks(p.dv);
    const void *fn = p.io_bf16 ? (kb == 2 ? pick<1, 2>(jb) : pick<1, 4>(jb)) : (kb == 2 ? pick<3, 2>(jb) : pick<3, 4>(jb));
    return hipLaunchKernel(fn, dim3((unsigned)p.nslot * p.Hk), dim3(512), args, 0, s);
}

}  // namespace gdr
