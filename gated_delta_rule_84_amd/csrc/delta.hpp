// delta.hpp -- launchers and device pieces of the trainable delta rule
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
// Products run on bf16 matrix cores: an fp32 operand is split into three bf16 terms that hold all of its 24 bits (bits cut,
// not rounded: the terms sum to it exactly), a bf16 one is its own only term.  The products of terms i, j with i + j < 3 are
// summed in fp32: with a bf16 operand that is all of them; of two fp32 ones the rest, of the product's own sign, is up to 2^-21
// of it and 2^-24.5 on the mean.  bf16 cores do such a product in 3/16 (one exact operand) to 6/16 of the time of the fp32 ones.
// Two terms (16 bits) are kept of operands that only a bf16 output reads, and of two such ones the products i + j < 2: up to
// 2^-15 of a product with a bf16 operand left out (2^-17 on the mean), 2^-13 of the others (2^-15.4), in 2/16 and 3/16 of
// the time; the output's own rounding is up to 2^-8.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "delta_place.hpp"
#include "gdr_device.hpp"
#include "gdr_mfma.hpp"

namespace gdr {

constexpr int kDeltaGates = 256;   // floats kept per (slot, value head), a fragment: front, behind * beta, whole
constexpr int kDeltaTri = 18;      // fragments of a triangular 64 x 64 matrix: 6 places of 3 terms

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
long delta_chain_threads(const DeltaParams &p);  // of the recurrence's launch
hipError_t launch_delta_fwd(const DeltaParams &p, hipStream_t s);
hipError_t launch_delta_bwd(const DeltaParams &p, hipStream_t s);
hipError_t launch_delta_prep(const DeltaParams &p, bool bwd, hipStream_t s);
hipError_t launch_delta_chain(const DeltaParams &p, bool bwd, hipStream_t s);
hipError_t launch_delta_grad(const DeltaParams &p, hipStream_t s);
hipError_t launch_delta_step(const DeltaStepParams &p, hipStream_t s);

// Tiles are 16 x 16: lane (r, q) has rows 4 q .. 4 q + 3 of column r, as the matrix cores leave a result.  A chunk's
// tiles lie by columns of the state, of each first those of the state's rows and then those of its 64 tokens.
// Row 4 q + i of tile a is channel 32 (a / 2) + 8 q + 4 (a % 2) + i: eight channels of a lane quarter in a row.
inline __host__ __device__ int delta_row_tiles(int dk) { return (dk + 31) / 32 * 2; }
inline __host__ __device__ int delta_col_tiles(int dv) { return (dv + 15) / 16; }
inline __host__ __device__ long delta_tiles(int dk, int dv) { return (long)delta_col_tiles(dv) * (delta_row_tiles(dk) + kDeltaC / 16); }

// Blocks of 32 channels that a kernel is built for.
inline int delta_blocks(int d) { return d <= 64 ? 2 : 4; }

namespace {

// Index of the 32-block of a contraction that element e of lane quarter q stands for: the rows of two
// accumulator tiles above each other, so that a product's result is the next one's operand as it lies.
__device__ __forceinline__ int perm(int q, int e) { return e < 4 ? 4 * q + e : 12 + 4 * q + e; }

// The upper halves of two fp32 values, cut, as a pair of bf16.
__device__ __forceinline__ uint32_t high_halves(float a, float b) {
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

// Eight fp32 values as NT bf16 terms.
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

// Elements 0 to 3 and 16 to 19 from there on: a lane's part of a block of 32 in the order of perm.
template <int NT>
__device__ __forceinline__ void load44(const void *base, long at, bool first, bool second, bf16x8 (&t)[NT]) {
    if constexpr (NT == 1) {
        typedef uint32_t wu2 __attribute__((ext_vector_type(2), aligned(2)));
        wu2 a = {0, 0}, b = {0, 0};
        if (first) a = *reinterpret_cast<const wu2 *>(static_cast<const uint16_t *>(base) + at);
        if (second) b = *reinterpret_cast<const wu2 *>(static_cast<const uint16_t *>(base) + at + 16);
        t[0] = as_bf16x8((u32x4){a[0], a[1], b[0], b[1]});
    } else {
        wu4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
        if (first) a = *reinterpret_cast<const wu4 *>(static_cast<const float *>(base) + at);
        if (second) b = *reinterpret_cast<const wu4 *>(static_cast<const float *>(base) + at + 16);
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = __uint_as_float(a[i]);
            x[4 + i] = __uint_as_float(b[i]);
        }
        split<NT>(x, t);
    }
}

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

// A barrier for what goes through shared memory: global memory is not waited for (__syncthreads waits for loads that are
// asked for ahead).
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

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

// Place in an operand's kilobyte of lane (r, q)'s 16 bytes, of k and q: the rows swapped about by quarters, for the
// transposing reads.
__device__ __forceinline__ int key_place(int r, int q) { return 16 * q + (r ^ 4 * q); }

__device__ __forceinline__ bf16x8 fragment(const char *base, long at, int lane) {
    return as_bf16x8(*reinterpret_cast<const u32x4 *>(base + at * 1024 + lane * 16));
}

__device__ __forceinline__ void put_fragment(char *base, long at, int lane, bf16x8 x) {
    *reinterpret_cast<u32x4 *>(base + at * 1024 + lane * 16) = __builtin_bit_cast(u32x4, x);
}

typedef __attribute__((address_space(3))) char *lds_bytes;
typedef __attribute__((address_space(3))) u32x2 *lds_u32x2;
typedef __attribute__((address_space(3))) u32x4 *lds_u32x4;

// A matrix of ROWS x COLS as NT terms in shared memory, [term][column][row], the 32-byte units of 16 rows swapped about so
// that eight columns lie in different banks.  A lane's place for all tiles of 16 rows is one offset: the tile's
// number changes bits of it that only the swap also holds.  The transposing LDS read makes operands of it whose
// contraction runs over the columns.
template <int ROWS, int NT, int COLS>
struct Staged {
    uint16_t x[NT][COLS][ROWS];
    static constexpr int kCol = 2 * ROWS, kTerm = COLS * kCol;
    static __device__ __forceinline__ uint32_t place(int j) { return j * kCol + ((ROWS == 64 ? j >> 1 & 3 : j & (ROWS / 16 - 1)) << 5); }
    __device__ __forceinline__ lds_bytes base() { return (lds_bytes)&x[0][0][0]; }
    // rows 4 q .. 4 q + 3 of a tile in column j, at put_place(j, q)
    static __device__ __forceinline__ uint32_t put_place(int j, int q) { return place(j) + 8 * q; }
    __device__ __forceinline__ void put(uint32_t at, int tile, f32x4 v) {
        lds_bytes to = base() + (at ^ (uint32_t)tile << 5);
        float r[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            *(lds_u32x2)(to + n * kTerm) = (u32x2){high_halves(r[0], r[1]), high_halves(r[2], r[3])};
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] -= __uint_as_float(__float_as_uint(r[i]) & 0xffff0000u);
        }
    }
    // a lane's part of a column from row 32 b on in the order of perm, at put_place(j, q)
    __device__ __forceinline__ void column(uint32_t at, int b, bf16x8 (&t)[NT]) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const u32x2 x = *(lds_u32x2)(base() + (at ^ (uint32_t)(2 * b) << 5) + n * kTerm);
            const u32x2 y = *(lds_u32x2)(base() + (at ^ (uint32_t)(2 * b + 1) << 5) + n * kTerm);
            t[n] = as_bf16x8((u32x4){x[0], x[1], y[0], y[1]});
        }
    }
    // rows 8 m .. 8 m + 7 of column j, put or got whole
    __device__ __forceinline__ void put8(int j, int m, const bf16x8 (&t)[NT]) {
#pragma unroll
        for (int n = 0; n < NT; ++n) *(lds_u32x4)(base() + (place(j) ^ (uint32_t)(m >> 1) << 5) + 16 * (m & 1) + n * kTerm) = __builtin_bit_cast(u32x4, t[n]);
    }
    __device__ __forceinline__ void get8(int j, int m, bf16x8 (&t)[NT]) {
#pragma unroll
        for (int n = 0; n < NT; ++n) t[n] = as_bf16x8(*(lds_u32x4)(base() + (place(j) ^ (uint32_t)(m >> 1) << 5) + 16 * (m & 1) + n * kTerm));
    }
    // the operand whose rows are channel tile a's (delta_row_tiles) of matrices with channels as rows, at key_get_place(r, q)
    static __device__ __forceinline__ uint32_t key_get_place(int r, int q) {
        return (place(4 * q + (r >> 2)) ^ (uint32_t)(r & 2) << 4) + 16 * (r & 1);
    }
    __device__ __forceinline__ void key_get(uint32_t at, int a, int b, bf16x8 (&t)[NT]) {
        lds_bytes from = base() + (at ^ (uint32_t)(a >> 1) << 6) + 8 * (a & 1) + b * 32 * kCol;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t)(from + n * kTerm)));
            const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t)(from + n * kTerm + 16 * kCol)));
            t[n] = as_bf16x8((u32x4){x[0], x[1], y[0], y[1]});
        }
    }
    // the operand whose rows are the 16 of a tile and whose contraction the 32 columns from 32 b on (perm), at get_place(r, q)
    static __device__ __forceinline__ uint32_t get_place(int r, int q) { return place(4 * q + (r >> 2)) + 8 * (r & 3); }
    __device__ __forceinline__ void get(uint32_t at, int tile, bf16x8 (&t)[NT], int b = 0) {
        lds_bytes from = base() + (at ^ (uint32_t)tile << 5) + b * 32 * kCol;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t)(from + n * kTerm)));
            const u32x2 c = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t)(from + n * kTerm + 16 * kCol)));
            t[n] = as_bf16x8((u32x4){a[0], a[1], c[0], c[1]});
        }
    }
};

// x of another lane.  The caller's own lane number goes in: the shuffle intrinsics' indices, which do not depend on it, are formed
// before loops and take registers over them.
__device__ __forceinline__ int of_lane(int x, int from) { return __builtin_amdgcn_ds_bpermute(4 * from, x); }
__device__ __forceinline__ float of_lane(float x, int from) { return __int_as_float(of_lane(__float_as_int(x), from)); }
__device__ __forceinline__ double of_lane(double x, int from) { return __hiloint2double(of_lane(__double2hiint(x), from), of_lane(__double2loint(x), from)); }

// The gates of a chunk, in shared memory.  P, here in units of ln 2, is summed in 64 bits: behind a strong decay the
// difference of two fp32 sums would have lost the weak ones.  A gate below kDeltaCut cuts: it adds nothing to P, and decays
// across it are 0 (as they are in fp32 whatever they multiply: |S| < 2^128, and 2^128 e^-256 < 2^-241).  Without the cut a
// gate of -1e30, a mask of the type's lowest value among them, would take every later one of the chunk out of P.  So
// |P| <= 64 * 256 log2 e < 2^15 but for growth, and differences are exact to 2^-37.  The difference is rounded once, so
// the hardware's 2^x is as exact as an fp32 e^x.
constexpr float kDeltaCut = -256.f;

struct ChunkGates {
    double P[kDeltaC];
    int cut[kDeltaC];
    float beta[kDeltaC], front[kDeltaC], behind[kDeltaC];
    float whole;

    static __device__ __forceinline__ float power(float x) { return __builtin_amdgcn_exp2f(x); }
    __device__ __forceinline__ float decay(int t, int s) const {
        const float e = power((float)(P[t] - P[s]));
        return cut[t] == cut[s] ? e : 0.f;
    }
};

// One wave; publish with a barrier.
__device__ __forceinline__ void make_gates(const DeltaParams &p, const Place &at, int hv, int lane, ChunkGates &c) {
    const bool there = lane < at.n;
    const long row = at.row0 + lane;
    const float g = there ? ld_elem(p.g, row * p.ldg + hv, p.gate_bf16) : 0.f;
    const bool cuts = g < kDeltaCut;
    double P = cuts ? 0.0 : (double)g * 1.4426950408889634;
    int cut = cuts;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double up = of_lane(P, lane - d);
        const int cu = of_lane(cut, lane - d);
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
    c.front[lane] = cut == 0 ? c.power((float)P) : 0.f;
    c.behind[lane] = cut == lc ? c.power((float)(last - P)) : 0.f;
    if (lane == 63) c.whole = lc == 0 ? c.power((float)P) : 0.f;
}

}  // namespace
}  // namespace gdr
