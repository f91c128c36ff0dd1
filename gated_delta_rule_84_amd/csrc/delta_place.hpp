// delta_place.hpp -- parameter block of the trainable delta rule and the chunks of its sequences.  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdr {

constexpr int kDeltaC = 64;        // tokens of a chunk

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
    int raw;         // k and q are copied to shared memory as they are (bf16, 16-byte aligned rows)
    char *kf, *qf;   // per (slot, key head), as operands: not used when raw
    char *tf, *pf;   // per (slot, value head), as operands: T and Q, or their transposes (backward)
    float *gates;
    float *back;  // like ckpt: the gradient of the state behind the chunk, and y
    float *sum;   // gradients of q and k of shared key heads while they are summed
};

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

}  // namespace
}  // namespace gdr
