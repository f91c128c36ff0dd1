// delta.hpp -- parameter block, launchers and device pieces of the trainable delta rule
// (delta_prep.hip, delta_chain.hip, delta_grad.hip, delta_step.hip; entry points in delta_api.hip).
// Not installed.
//
// One sequence of one value head, in chunks of 64 tokens (row vectors k_t, q_t, v_t; S is dk x dv).
// With P_t the sum of the log gates of the chunk's tokens up to t,
//     front_t = e^{P_t}, e_ts = e^{P_t - P_s}, behind_s = e^{P_63 - P_s}, whole = e^{P_63}
//     A_ts = e_ts beta_s k_t.k_s (t > s),   T = (I + A)^{-1},   Q_ts = e_ts beta_s q_t.k_s (t >= s)
//     D = T (v - front k S)                 what the tokens write, before beta
//     o = front q S + Q D
//     S' = whole S + k^T (behind beta D)
// and from do and the gradient G of S', with y the gradient of v - front k S,
//     y = T^T (Q^T do + behind beta k G),   dv = y
//     dS = whole G + q^T (front do) - k^T (front y)
//
// Products run on bf16 matrix cores and lose nothing: an fp32 operand is split into three bf16
// terms that hold all of its 24 bits (bits cut, not rounded: the terms sum to it exactly), a bf16 one
// is its own only term.  The products of terms i, j with i + j < 3 are summed in fp32; what is left out
// is about 2^-24 of the result.  bf16 cores do such a product in 3/16 (one exact operand) to 6/16 of
// the time of the fp32 ones.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdr_device.hpp"
#include "gdr_mfma.hpp"

namespace gdr {

constexpr int kDeltaC = 64;        // tokens of a chunk
constexpr int kDeltaGates = 256;   // floats kept per (slot, value head), a fragment: front, behind * beta, whole
constexpr int kDeltaTri = 18;      // fragments of a triangular 64 x 64 matrix: 6 places of 3 terms

// Parameters of one call, already validated by the entry points.
struct DeltaParams {
    int B, T, Hk, Hv, dk, dv, group;
    int io_bf16, gate_bf16;
    const void *q, *k, *v, *g, *b;
    int64_t ldq, ldk, ldv, ldg, ldb;  // elements between tokens
    const int32_t *off;               // [nseq + 1] or NULL: borders of packed sequences
    int nseq;                         // sequences (B when dense)
    int chunks;                       // dense: chunks of a sequence
    int nslot;                        // chunk slots of the call
    const float *S0;
    void *o;
    float *ST;
    float *ckpt;  // per (slot, value head) the tiles of the state before the chunk and of its D; NULL: not kept
    const void *dout;
    const float *dST;
    void *dq, *dkk, *dvv, *dg, *db;
    float *dS0;
    // workspace
    char *kf, *ktf, *qf, *qtf;  // per (slot, key head)
    char *tf, *pf;              // per (slot, value head): T and Q, or their transposes (backward)
    float *gates;
    float *back;  // like ckpt: the gradient of the state behind the chunk, and y
    float *sum;   // gradients of q and k of shared key heads while they are summed
};

// Parameters of a single-token step.
struct DeltaStepParams {
    int B, Hk, Hv, dk, dv, group;
    int io_bf16, gate_bf16;
    const void *q, *k, *v, *g, *b;
    int64_t ldq, ldk, ldv, ldg, ldb;
    float *S;
    void *o;
};

// Bytes of the workspace, and the pointers into it.
size_t delta_workspace(DeltaParams &p, bool bwd, char *base);
hipError_t launch_delta_fwd(const DeltaParams &p, hipStream_t s);
hipError_t launch_delta_bwd(const DeltaParams &p, hipStream_t s);
hipError_t launch_delta_prep(const DeltaParams &p, bool bwd, hipStream_t s);
hipError_t launch_delta_chain(const DeltaParams &p, bool bwd, hipStream_t s);
hipError_t launch_delta_grad(const DeltaParams &p, hipStream_t s);
hipError_t launch_delta_step(const DeltaStepParams &p, hipStream_t s);

// Tiles are 16 x 16: lane (r, q) has rows 4 q .. 4 q + 3 of column r, as the matrix cores leave a result.  A chunk's
// tiles lie by columns of the state, of each first those of the state's rows and then those of its 64 tokens.
inline __host__ __device__ int delta_row_tiles(int dk) { return (dk + 15) / 16; }
inline __host__ __device__ int delta_col_tiles(int dv) { return (dv + 15) / 16; }
inline __host__ __device__ long delta_tiles(int dk, int dv) { return (long)delta_col_tiles(dv) * (delta_row_tiles(dk) + kDeltaC / 16); }

// Blocks of 32 channels that a kernel is built for.
inline int delta_blocks(int d) { return d <= 64 ? 2 : 4; }

namespace {

// Where a slot lies: the rows row0 .. row0 + n - 1 (of B * T) of sequence seq; n <= 0 for none.  Sequence i
// of a packed call takes the slots from off[i] / 64 + i on, which no other sequence reaches; offsets are
// held inside 0 .. T, so that no access passes the tensors whatever they are.
struct Place {
    int seq, n;
    long row0;
};

__device__ __forceinline__ int offset_at(const DeltaParams &p, int i) { return min(max(p.off[i], 0), p.T); }

__device__ __forceinline__ int first_slot(const DeltaParams &p, int seq) {
    return p.off ? offset_at(p, seq) / kDeltaC + seq : seq * p.chunks;
}

// Tokens and the first row of a sequence.
__device__ __forceinline__ int tokens_of(const DeltaParams &p, int seq, long &row0) {
    if (!p.off) {
        row0 = (long)seq * p.T;
        return p.T;
    }
    const int a = offset_at(p, seq), b = offset_at(p, seq + 1);
    row0 = a;
    return b > a ? b - a : 0;
}

__device__ __forceinline__ Place place_of(const DeltaParams &p, int slot) {
    Place r;
    if (p.off) {
        int lo = 0, hi = p.nseq - 1;  // the last sequence whose first slot is not behind this one
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first_slot(p, mid) <= slot) lo = mid;
            else hi = mid - 1;
        }
        r.seq = lo;
    } else {
        r.seq = slot / p.chunks;
    }
    long start;
    const int len = tokens_of(p, r.seq, start), c = slot - first_slot(p, r.seq);
    r.row0 = start + (long)c * kDeltaC;
    r.n = c < 0 ? 0 : min(kDeltaC, len - c * kDeltaC);
    return r;
}

// Index of the 32-block of a contraction that element e of lane quarter q stands for: the rows of two
// accumulator tiles above each other, so that a product's result is the next one's operand as it lies.
__device__ __forceinline__ int perm(int q, int e) { return e < 4 ? 4 * q + e : 12 + 4 * q + e; }

// Eight fp32 values as three bf16 terms.
struct Split3 {
    bf16x8 t[3];
};

__device__ __forceinline__ uint32_t high_halves(float a, float b) {
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

template <int NT>
__device__ __forceinline__ void split(const float (&x)[8], bf16x8 (&t)[NT]) {
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = x[e];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 8; e += 2) w[e / 2] = high_halves(r[e], r[e + 1]);
        t[n] = as_bf16x8(w);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (n + 1 < NT) r[e] -= __uint_as_float(__float_as_uint(r[e]) & 0xffff0000u);
    }
}

// two accumulator tiles above each other
template <int NT>
__device__ __forceinline__ void split(f32x4 lo, f32x4 hi, bf16x8 (&t)[NT]) {
    const float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    split<NT>(x, t);
}

// acc[k] += A[k] B[k] over one 32-block for K results, terms i and j with i + j < the larger count, the smallest first.
// Term by term over all results: a matrix instruction that adds to what the one before it gives would wait for it.
template <int NA, int NB, int K, class A, class B, class C>
__device__ __forceinline__ void products(A &&a, B &&b, C &&acc) {
    constexpr int N = NA > NB ? NA : NB;
#pragma unroll
    for (int s = N - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB) {
#pragma unroll
                for (int k = 0; k < K; ++k) acc(k) = mfma(a(k, i), b(k, s - i), acc(k));
            }
}

template <int NA, int NB>
__device__ __forceinline__ f32x4 product(const bf16x8 (&a)[NA], const bf16x8 (&b)[NB], f32x4 acc) {
    products<NA, NB, 1>([&](int, int i) { return a[i]; }, [&](int, int j) { return b[j]; }, [&](int) -> f32x4 & { return acc; });
    return acc;
}

// Eight elements at an element-aligned address (the hardware takes a global access of a dword or
// more at any byte address) as terms: bf16 as they are, fp32 split.
typedef uint32_t wu4 __attribute__((ext_vector_type(4), aligned(2)));

template <int NT>
__device__ __forceinline__ void load8(const void *base, long at, bool there, bf16x8 (&t)[NT]) {
    if constexpr (NT == 1) {
        wu4 w = {0, 0, 0, 0};
        if (there) w = *reinterpret_cast<const wu4 *>(static_cast<const uint16_t *>(base) + at);
        t[0] = as_bf16x8((u32x4){w[0], w[1], w[2], w[3]});
    } else {
        float x[8];
        wu4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
        if (there) {
            a = *reinterpret_cast<const wu4 *>(static_cast<const float *>(base) + at);
            b = *reinterpret_cast<const wu4 *>(static_cast<const float *>(base) + at + 4);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = __uint_as_float(a[i]);
            x[4 + i] = __uint_as_float(b[i]);
        }
        split<NT>(x, t);
    }
}

// A range-checked buffer: loads from outside give 0, stores to outside are dropped.  A lane that is
// to be left out adds kNowhere to its offset.
typedef __amdgpu_buffer_rsrc_t Buf;
constexpr uint32_t kNowhere = 0x7ff00000u;

__device__ __forceinline__ Buf buffer(const void *base, long bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, (int)bytes, 0x00020000);
}

// An element's bits, to be made a number where it is used: made one here, it would be waited for here.
template <bool BF>
__device__ __forceinline__ uint32_t load1(Buf b, uint32_t at) {
    if constexpr (BF) return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(b, at, 0, 0);
    return __builtin_amdgcn_raw_buffer_load_b32(b, at, 0, 0);
}

template <bool BF>
__device__ __forceinline__ float number(uint32_t bits) { return __uint_as_float(BF ? bits << 16 : bits); }

template <bool BF>
__device__ __forceinline__ void store1(Buf b, uint32_t at, float x) {
    if constexpr (BF) __builtin_amdgcn_raw_buffer_store_b16((uint16_t)pk_bf16(x, x), b, at, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), b, at, 0, 0);
}

__device__ __forceinline__ bf16x8 fragment(const char *base, long at, int lane) {
    return as_bf16x8(*reinterpret_cast<const u32x4 *>(base + at * 1024 + lane * 16));
}

__device__ __forceinline__ void put_fragment(char *base, long at, int lane, bf16x8 x) {
    *reinterpret_cast<u32x4 *>(base + at * 1024 + lane * 16) = __builtin_bit_cast(u32x4, x);
}

// The gates of a chunk, in shared memory.  P is summed in 64 bits: behind a strong decay the
// difference of two fp32 sums would have lost the weak ones.  A gate of -inf cuts: it adds nothing to P,
// and decays across it are 0.
struct ChunkGates {
    double P[kDeltaC];
    int cut[kDeltaC];
    float beta[kDeltaC], front[kDeltaC], behind[kDeltaC];
    float whole;

    __device__ __forceinline__ float decay(int t, int s) const {
        return cut[t] == cut[s] ? expf((float)(P[t] - P[s])) : 0.f;
    }
};

// One wave; publish with a barrier.
__device__ __forceinline__ void make_gates(const DeltaParams &p, const Place &at, int hv, int lane, ChunkGates &c) {
    const bool there = lane < at.n;
    const long row = at.row0 + lane;
    const float g = there ? ld_elem(p.g, row * p.ldg + hv, p.gate_bf16) : 0.f;
    const bool cuts = g == -INFINITY;
    double P = cuts ? 0.0 : (double)g;
    int cut = cuts;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double up = __shfl_up(P, d);
        const int cu = __shfl_up(cut, d);
        if (lane >= d) {
            P += up;
            cut += cu;
        }
    }
    const double last = __shfl(P, 63);
    const int lc = __shfl(cut, 63);
    c.P[lane] = P;
    c.cut[lane] = cut;
    c.beta[lane] = there ? ld_elem(p.b, row * p.ldb + hv, p.gate_bf16) : 0.f;
    c.front[lane] = cut == 0 ? expf((float)P) : 0.f;
    c.behind[lane] = cut == lc ? expf((float)(last - P)) : 0.f;
    if (lane == 63) c.whole = lc == 0 ? expf((float)P) : 0.f;
}

}  // namespace
}  // namespace gdr
