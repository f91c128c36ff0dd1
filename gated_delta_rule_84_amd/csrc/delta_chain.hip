// delta_chain.hip -- the recurrence of the delta rule over a sequence's chunks, forward and backward (delta.hpp).
#include <type_traits>

#include "delta.hpp"

namespace gdr {
namespace {

constexpr int kLoaders = 2;   // waves that copy
constexpr int kGroup = 12;    // most fragments that a wave reads ahead

__device__ const u32x4 kNothing = {0, 0, 0, 0};  // what is copied for rows and channels that are not there

// 4 bytes per lane, global -> LDS; lane l writes dst + 4 l.
__device__ __forceinline__ void dma4(const void *src, void *dst) {
    __builtin_amdgcn_global_load_lds((gbl_void_t)src, (lds_void_t)dst, 4, 0, 0);
}

// until at most so many of this wave's loads, the last ones, are under way (or 2, if more)
__device__ __forceinline__ void wait_copies(int n) {
    if (n == 0) __builtin_amdgcn_s_waitcnt(0x0F70);
    else if (n == 1) __builtin_amdgcn_s_waitcnt(0x0F71);
    else __builtin_amdgcn_s_waitcnt(0x0F72);
}

template <int I, int N, class F>
__device__ __forceinline__ void each(F &&f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>());
        each<I + 1, N>(f);
    }
}

// Places (16-row tile, 32-column block) of triangular operands: the six that are not zero.
template <bool UPPER>
constexpr int tri_index(int a, int b) {
    return UPPER ? (a < 2 ? 2 * a + b : b == 1 ? a + 2 : -1) : (a < 2 ? (b == 0 ? a : -1) : 2 * a - 2 + b);
}

// Groups of products, by the operand that they read from shared memory.
enum Part { kK, kQ, kT, kP, kC, kQC };  // k, q, T, Q (their transposes in the backward pass), k^T, q^T

template <int NT, int KB, bool BWD, int SPLIT>
struct Plan {
    static constexpr int L = KB / SPLIT;  // blocks of channels of a wave
    // a chunk's operands in shared memory, in fragments of 1 KB: k, q, T, Q
    static constexpr int key = 4 * KB * NT, atQ = key, atT = 2 * key, atP = atT + kDeltaTri;
    static constexpr int nP = BWD || NT == 3 ? 3 : 2, size = atP + 6 * nP;  // terms of Q: forward, only o reads it
    static constexpr int sets = NT == 1 ? 2 : 1;  // chunks at once
    // groups: of k a block of channels, of q GQ blocks, of T and Q a block of their columns, of k^T and q^T GC tiles of
    // channels.  Backward with bf16, q^T's second half comes behind T: products beside the splits that T's result needs.
    static constexpr int GQ = NT == 1 && L > 1 ? 2 : 1, GC = NT == 1 || L == 1 ? 2 * L : 4;
    static constexpr int nQ = L / GQ, nC = 4 * L / GC, late = BWD && NT == 1 ? nC / 2 : 0;
    static constexpr int groups = BWD ? 2 + L + nC + 2 + nC : L + nQ + 2 + 2 + nC;
    struct At {
        Part x;
        int g;
    };
    static constexpr At at(int i) {
        // forward with bf16, the products that only o needs come last, beside the splits of the next chunk's first operands
        const Part f[] = {kK, kQ, kT, NT == 1 ? kC : kP, NT == 1 ? kP : kC}, b[] = {kP, kK, kQC, kT, kQC, kC};
        const int nf[] = {L, nQ, 2, NT == 1 ? nC : 2, NT == 1 ? 2 : nC}, nb[] = {2, L, nC - late, 2, late, nC};
        for (int s = 0; s < (BWD ? 6 : 5); ++s) {
            const int n = BWD ? nb[s] : nf[s];
            if (i < n) return {BWD ? b[s] : f[s], i + (BWD && s == 4 ? nC - late : 0)};
            i -= n;
        }
        return {kK, 0};
    }
};

// A workgroup has NW / SPLIT tiles of 16 columns of one value head's state, in registers: of each one wave has all rows, or
// two waves half of the channels each.  Every product's result is the next one's operand as it lies (perm in delta.hpp), so
// waves of one tile exchange nothing; two of them exchange their parts of k S and q S, and both form what follows from the
// sums.  Two more waves copy the operands, which the tiles share, to shared memory: with bf16 a chunk ahead, with
// fp32, whose operands are three times as large, as soon as the chunk before is done with a part.
//
// What bounds it: chunks come one after the other, each a chain of products (k S, T R, k^T E) and of splits between
// them, with one wave to a SIMD.  4 x 4,096 tokens, 16 heads of 128 x 128, bf16: 176 us at best, 200 on the mean (64 chunks of 2.8
// us; the matrix cores' part is 0.8), 157 with nothing copied; with what the backward pass needs 217 (0.46 GB written, 3.7 TB/s in
// all), the backward pass 232.
// KEEP: the states before the chunks and E are stored, for the backward pass.
template <int NT, int KB, bool BWD, bool KEEP, int NW, int SPLIT>
__global__ void __launch_bounds__(64 * (NW + kLoaders)) delta_chain_kernel(DeltaParams p, int heads8) {
    constexpr int NX = NT == 1 ? 2 : 3;  // terms of what only outputs of the io type read
    typedef Plan<NT, KB, BWD, SPLIT> P;
    constexpr bool HOLD = SPLIT == 2 && NT == 1;  // gates in registers: read where they are needed, they are waited for
    constexpr int L = P::L, NO = SPLIT == 2 ? 2 : 4;  // NO: tiles of tokens whose results a wave stores
    __shared__ __attribute__((aligned(16))) char sets[P::sets][P::size * 1024];
    __shared__ __attribute__((aligned(16))) float gring[2][kDeltaGates], nowhere[64];
    __shared__ f32x4 halves[SPLIT == 2 ? NW : 1][4][64], halves_o[SPLIT == 2 && !BWD ? NW : 1][2][64];
    __shared__ int given[NW], given_o[NW];  // chunks whose sums a wave has given to the other half's
    const int head = blockIdx.x % heads8;
    if (head >= p.nseq * p.Hv) return;  // uniform over the workgroup
    const int seq = head / p.Hv, hv = head % p.Hv, hk = hv / p.group;
    long row0;
    const int len = tokens_of(p, seq, row0), nc = (len + kDeltaC - 1) / kDeltaC;
    const int slot0 = first_slot(p, seq);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, r = l & 15, q = l >> 4;

    if (w >= NW) {  // a copying wave has every second fragment
        const int half = w - NW;
        // of chunk number c in the order of the pass: k and the gates (first), the rest
        auto copy = [&](int c, bool first, bool rest) __attribute__((always_inline)) {
            const int pos = BWD ? nc - 1 - c : c, n = len - pos * kDeltaC;
            const long slot = slot0 + pos, kh = slot * p.Hk + hk, vh = slot * p.Hv + hv;
            char *to = sets[P::sets == 2 ? c & 1 : 0];
            auto keys = [&](const void *x, int64_t ld, const char *made, int at) __attribute__((always_inline)) {
                if (NT == 1 && p.raw) {  // lane's place: row pr, channels from 8 q on
                    const int pr = r ^ 4 * q;
                    const uint16_t *from = static_cast<const uint16_t *>(x) + (row0 + (long)pos * kDeltaC + pr) * ld + (long)hk * p.dk + 8 * q;
#pragma unroll
                    for (int f = 0; f < P::key; f += kLoaders) {
                        const int i = f + half, a = i & 3, kb = i >> 2;
                        const bool there = 16 * a + pr < n && 32 * kb + 8 * q < p.dk;
                        dma16(there ? static_cast<const void *>(from + 16 * a * ld + 32 * kb) : &kNothing, to + (at + i) * 1024);
                    }
                } else {
                    const char *from = made + (kh * P::key + half) * 1024 + l * 16;
#pragma unroll 8
                    for (int f = 0; f < P::key; f += kLoaders) dma16(from + f * 1024, to + (at + half + f) * 1024);
                }
            };
            if (first) {
                keys(p.k, p.ldk, p.kf, 0);
                if (half) dma16(reinterpret_cast<const char *>(p.gates + vh * kDeltaGates) + l * 16, gring[c & 1]);
            }
            if (rest) {
                keys(p.q, p.ldq, p.qf, P::atQ);
                const char *t = p.tf + (vh * kDeltaTri + half) * 1024 + l * 16, *s = p.pf + (vh * kDeltaTri + half) * 1024 + l * 16;
#pragma unroll
                for (int f = 0; f < kDeltaTri; f += kLoaders) dma16(t + f * 1024, to + (P::atT + half + f) * 1024);
#pragma unroll
                for (int f = 0; f < 6 * P::nP; f += kLoaders) dma16(s + f * 1024, to + (P::atP + half + f) * 1024);
            }
        };
        // Brings chunk c's operands to the XCD's cache: 4 bytes of every 128-byte line, to nowhere.  The workgroups of a head
        // share the work.
        const int parts = gridDim.x / heads8, part = blockIdx.x / heads8;
        auto touch = [&](int c) __attribute__((always_inline)) {
            const int pos = BWD ? nc - 1 - c : c, n = len - pos * kDeltaC;
            const long slot = slot0 + pos, kh = slot * p.Hk + hk, vh = slot * p.Hv + hv;
            int issued = 0;
            auto lines = [&](const char *from, int bytes) __attribute__((always_inline)) {
                for (int i = half * 8192; i < bytes; i += kLoaders * 8192, ++issued) dma4(from + min(i + l * 128, bytes - 128), nowhere);
            };
            auto keys = [&](const void *x, int64_t ld, const char *made) __attribute__((always_inline)) {
                if (NT == 1 && p.raw) {
                    const int row = min(l, n - 1), ch = min(64 * half, p.dk - 8);  // 128 bytes of each row a wave
                    dma4(static_cast<const uint16_t *>(x) + (row0 + (long)pos * kDeltaC + row) * ld + (long)hk * p.dk + ch, nowhere);
                    ++issued;
                } else {
                    lines(made + kh * P::key * 1024, P::key * 1024);
                }
            };
            if (part == 0) keys(p.k, p.ldk, p.kf);
            if (part == min(1, parts - 1)) keys(p.q, p.ldq, p.qf);
            if (part == min(2, parts - 1)) lines(p.tf + vh * kDeltaTri * 1024, kDeltaTri * 1024);
            if (part == min(3, parts - 1)) lines(p.pf + vh * kDeltaTri * 1024, 6 * P::nP * 1024);
            return issued;
        };
        if (nc > 0) copy(0, true, true);
        int young = nc > 1 ? touch(1) : 0;  // touches behind the last copy, which are not waited for
        for (int c = 0; c < nc; ++c) {
            wait_copies(young);  // this chunk's are there
            young = 0;
            lds_barrier();  // and the chunk before is done
            if constexpr (P::sets == 2) {
                if (c + 1 < nc) copy(c + 1, true, true);
                if (c + 2 < nc) young = touch(c + 2);
            } else {
                lds_barrier();  // q, T and Q are no longer read
                if (c + 1 < nc) copy(c + 1, false, true);
                lds_barrier();  // nor is k
                if (c + 1 < nc) copy(c + 1, true, false);
                if (c + 2 < nc) young = touch(c + 2);
            }
        }
        return;
    }

    const int h = SPLIT == 2 ? w & 1 : 0;  // half of the channels
    if constexpr (SPLIT == 2) given[w] = given_o[w] = 0;
    const int tile = (int)(blockIdx.x / heads8) * (NW / SPLIT) + w / SPLIT, na = delta_row_tiles(p.dk), nj = delta_col_tiles(p.dv);
    const int col = 16 * tile + r;
    const bool mine = col < p.dv;
    const long sstate = (long)p.dk * p.dv;
    // accesses by tiles go through range-checked buffers: no branch per element for rows and channels that are not there
    constexpr bool BF = NT == 1;
    constexpr int es = BF ? 2 : 4;
    const uint32_t away = mine ? 0 : kNowhere, srow = 4 * p.dv, sat = (32 * L * h + 8 * q) * srow + 4 * col + away;
    auto channel = [](int a, int i) { return 32 * (a / 2) + 4 * (a % 2) + i; };  // of a tile's row, from 8 q on
    auto keep = [&](float *to, const f32x4 (&S)[2 * L]) __attribute__((always_inline)) {
        const Buf b = buffer(to, 4 * sstate);
#pragma unroll
        for (int a = 0; a < 2 * L; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) store1<false>(b, sat + channel(a, i) * srow, S[a][i]);
    };
    f32x4 S[2 * L];
    {
        const float *init = BWD ? p.dST : p.S0;
        const Buf b = buffer(init + (init ? head * sstate : 0), init ? 4 * sstate : 0);
#pragma unroll
        for (int a = 0; a < 2 * L; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[a][i] = number<false>(load1<false>(b, sat + channel(a, i) * srow));
    }
    // v, or do, of the lane's rows 16 a + 4 q + i of a chunk
    const int64_t ldx = BWD ? (int64_t)p.Hv * p.dv : p.ldv;
    const uint32_t xrow = ldx * es, orow = (uint32_t)p.Hv * p.dv * es;
    auto values = [&](int c, uint32_t (&x)[4][4]) __attribute__((always_inline)) {
        const int n = min(kDeltaC, len - c * kDeltaC);
        const char *from = static_cast<const char *>(BWD ? p.dout : p.v) + ((row0 + (long)c * kDeltaC) * ldx + (long)hv * p.dv) * es;
        const Buf b = buffer(from, (long)(n - 1) * xrow + p.dv * es);
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[a][i] = load1<BF>(b, 4 * q * xrow + es * col + away + (16 * a + i) * xrow);
    };
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    uint32_t x_[4][4];
    auto value = [&](int a) __attribute__((always_inline)) -> f32x4 {
        return (f32x4){number<BF>(x_[a][0]), number<BF>(x_[a][1]), number<BF>(x_[a][2]), number<BF>(x_[a][3])};
    };
    bf16x8 sf[L][3], df[2][NT];
    auto ahead = [&]() __attribute__((always_inline)) {  // the first operands of a chunk
        split<3>(S[0], S[1], sf[0]);
        if constexpr (BWD) {
            split<NT>(value(0), value(1), df[0]);
            split<NT>(value(2), value(3), df[1]);
        }
    };
    if (nc > 0) {
        values(BWD ? nc - 1 : 0, x_);
        ahead();
        // As many stores, dropped ones, as a chunk has behind its loads of values: at the top of the loop the compiler has one
        // count of what is under way, and without them it waits for a chunk's stores together with its values.
        if constexpr (!BWD && NT == 1) {
            const Buf none = buffer(nullptr, 0);
#pragma unroll
            for (int a = 0; a < 4 * NO; ++a) store1<BF>(none, 64 * a, 0.f);
            if constexpr (KEEP) {
#pragma unroll
                for (int a = 0; a < NO; ++a) __builtin_amdgcn_raw_buffer_store_b128((u32x4){0, 0, 0, 0}, none, 64 * a, 0, 0);
            }
        }
    }
    for (int cc = 0; cc < nc; ++cc) {
        const int c = BWD ? nc - 1 - cc : cc;
        const int n = min(kDeltaC, len - c * kDeltaC);
        const long vh = (long)(slot0 + c) * p.Hv + hv, row = row0 + (long)c * kDeltaC;
        const float *gates = gring[cc & 1] + 4 * q;
        const char *ops = sets[P::sets == 2 ? cc & 1 : 0];
        const int keyl = key_place(r, q);
        const lds_bytes ctl = (lds_bytes)(char *)ops + key_place(4 * q + (r >> 2), r & 3) * 16;  // of the transposing reads
        auto gate = [&](int a) __attribute__((always_inline)) { return *reinterpret_cast<const f32x4 *>(gates + 16 * a); };
        f32x4 held[HOLD ? 8 : 1], held_o[HOLD ? 2 : 1];
        auto front = [&](int a) __attribute__((always_inline)) { return HOLD ? held[a] : gate(a); };
        auto wb = [&](int a) __attribute__((always_inline)) { return HOLD ? held[4 + a] : gate(4 + a); };
        // token tile of which a wave has the j-th rows: split, two whose triangular rows are as long as the other two's
        auto mine_of = [&](int j) __attribute__((always_inline)) { return SPLIT == 1 ? j : j == 0 ? h : j == 1 ? 3 - h : j == 2 ? 1 - h : 2 + h; };
        f32x4 R[4] = {zero, zero, zero, zero}, E[4] = {zero, zero, zero, zero};
        f32x4 O[4] = {zero, zero, zero, zero};  // o; backward: Q^T do
        bf16x8 rf[2][3], ef[2][3], of[2][NX], xf[2][3];
        // tiles are kept as they lie: 16 bytes a lane (by elements of rows, 48 stores a chunk, their acknowledgements
        // held the wave up)
        auto tiles = [&](int n) __attribute__((always_inline)) {
            return buffer((BWD ? p.back : p.ckpt) + (vh * nj + tile) * (na + kDeltaC / 16) * 256, tile < nj ? n * 1024 : 0);
        };
        auto put_tile = [&](Buf b, int a, f32x4 x) __attribute__((always_inline)) {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), b, a * 1024 + l * 16, 0, 0);
        };
        // Split, a wave's products with the state sum over its channels only.  The two waves of a tile exchange such sums by
        // themselves: a barrier would wait for the copying waves.  A wave's accesses to shared memory are done in order: what it
        // writes before a count is there when the count is, and a count read before the sums says whether they were.
        auto give = [&](int *count, f32x4 (*to)[64], const f32x4 *x, int n) __attribute__((always_inline)) {
#pragma unroll
            for (int a = 0; a < n; ++a) to[a][l] = x[a];
            asm volatile("" ::: "memory");
            count[w] = cc + 1;
            asm volatile("" ::: "memory");
        };
        auto take = [&](int *count, f32x4 (*from)[64], f32x4 *x, int n) __attribute__((always_inline)) {
            f32x4 y[4];
            for (bool there = false; !there;) {  // the other wave gives its sums before it waits for these
                const int seen = count[w ^ 1];
                asm volatile("" ::: "memory");
#pragma unroll
                for (int a = 0; a < n; ++a) y[a] = from[a][l];
                asm volatile("" ::: "memory");
                there = __builtin_amdgcn_readfirstlane(seen) > cc;
            }
#pragma unroll
            for (int a = 0; a < n; ++a) x[a] += y[a];  // a sum of two is the same in both waves
        };
        auto mine_e = [&](int j) __attribute__((always_inline)) -> f32x4 {
            if constexpr (SPLIT == 1) return E[j];
            return j == 0 ? (h ? E[1] : E[0]) : (h ? E[2] : E[3]);
        };
        auto decay = [&]() __attribute__((always_inline)) {
            const float whole = gring[cc & 1][128];
#pragma unroll
            for (int a = 0; a < 2 * L; ++a) S[a] = whole * S[a];
        };
        auto put_tokens = [&]() __attribute__((always_inline)) {  // E
            const Buf b = tiles(na + kDeltaC / 16);
#pragma unroll
            for (int a = 0; a < NO; ++a) put_tile(b, na + mine_of(a), mine_e(a));
        };
        auto put_rows = [&]() __attribute__((always_inline)) {  // o, or dv
            char *to = static_cast<char *>(BWD ? p.dvv : p.o) + (row * p.Hv + hv) * p.dv * es;
            const Buf b = buffer(to, (long)(n - 1) * orow + p.dv * es);
#pragma unroll
            for (int a = 0; a < NO; ++a) {
                const f32x4 y = BWD ? mine_e(a) : O[a];
#pragma unroll
                for (int i = 0; i < 4; ++i) store1<BF>(b, 4 * q * orow + es * col + away + (16 * mine_of(a) + i) * orow, y[i]);
            }
        };
        // T^T goes by its second block first: rows 32 to 63 of the result are done with it, as forward rows 0 to 31 with the first
        constexpr auto tri_block = [](Part x, int g) { return BWD && x == kT ? 1 - g : g; };
        // reads the fragments of group G
        auto load = [&](auto G, bf16x8 (&to)[kGroup]) __attribute__((always_inline)) {
            constexpr Part x = P::at(G).x;
            constexpr int g = P::at(G).g;
            if constexpr (P::sets == 1 && x == kC && g == 0) lds_barrier();  // q, T and Q are no longer read
            if constexpr (x == kT || x == kP) {
                constexpr int NF = x == kP ? P::nP : 3, at = x == kT ? P::atT : P::atP;
                if constexpr (SPLIT == 2 && !BWD && x == kP) {  // tile h, which has the first block only, and tile 3 - h
#pragma unroll
                    for (int k = 0; k < 2 - g; ++k)
#pragma unroll
                        for (int n = 0; n < NF; ++n) to[k * NF + n] = fragment(ops, at + n + NF * (k + g == 0 ? h : 4 - 2 * h + g), l);
                    return;
                }
                constexpr int tb = tri_block(x, g), t0 = BWD ? 0 : 2 * tb, nt = BWD ? 2 + 2 * tb : 4 - 2 * tb;
#pragma unroll
                for (int k = 0; k < nt; ++k)
#pragma unroll
                    for (int n = 0; n < NF; ++n) to[k * NF + n] = fragment(ops, at + NF * tri_index<BWD>(t0 + k, tb) + n, l);
            } else if constexpr (x == kK || x == kQ) {
                constexpr int n = (x == kK ? 4 : 4 * P::GQ) * NT, at = (x == kK ? 0 : P::atQ) + g * n;
                const int mine = at + h * L * 4 * NT;
#pragma unroll
                for (int k = 0; k < n; ++k) to[k] = fragment(ops, x == kK ? mine + k : mine + k / (4 * NT) * 4 * NT + mine_of(k / NT % 4) * NT + k % NT, keyl);
            } else {
#pragma unroll
                for (int k = 0; k < P::GC; ++k)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        constexpr int b = g * P::GC / (2 * L);
                        const int a = (g * P::GC + k) % (2 * L);
                        const int at = (x == kC ? 0 : P::atQ) + ((h * L + a / 2) * 4 + 2 * b) * NT + n;
                        const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t)(ctl + at * 1024 + 8 * (a & 1))));
                        const u32x2 z = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t)(ctl + (at + NT) * 1024 + 8 * (a & 1))));
                        to[k * NT + n] = as_bf16x8((u32x4){y[0], y[1], z[0], z[1]});
                    }
            }
        };
        // the products of group G, and beside them the operands of later groups
        auto run = [&](auto G, const bf16x8 (&from)[kGroup]) __attribute__((always_inline)) {
            constexpr Part x = P::at(G).x;
            constexpr int g = P::at(G).g;
            constexpr int tb = tri_block(x, g), t0 = BWD ? 0 : 2 * tb, nt = BWD ? 2 + 2 * tb : 4 - 2 * tb;  // a triangle's block, its row tiles
            if constexpr (x == kK) {  // R = k S
                products<NT, 3, 4>([&](int k, int i) { return from[k * NT + i]; }, [&](int, int j) { return sf[g][j]; },
                                   [&](int k) -> f32x4 & { return R[k]; });
                if constexpr (g + 1 < L) split<3>(S[2 * g + 2], S[2 * g + 3], sf[g + 1]);
                if constexpr (g == 0) {
                    if constexpr (KEEP) {
                        const Buf b = tiles(na);  // tiles past dk are dropped
#pragma unroll
                        for (int a = 0; a < 2 * L; ++a) put_tile(b, 2 * L * h + a, S[a]);
                    }
                }
                if constexpr (BWD && g == L - 1) decay();
            } else if constexpr (x == kQ) {  // O = q S
                if constexpr (SPLIT == 2 && g == 0) give(given, halves[w], R, 4);
                products<NT, NX, 4 * P::GQ>([&](int k, int i) { return from[k * NT + i]; },
                                            [&](int k, int j) { return sf[g * P::GQ + k / 4][j]; },
                                            [&](int k) -> f32x4 & { return O[k % 4]; });
                if constexpr (SPLIT == 2 && g == P::nQ - 1) {
                    give(given_o, halves_o[w], O + 2, 2);
                    take(given, halves[w ^ 1], R, 4);
                }
                if constexpr (g == (SPLIT == 2 ? P::nQ - 1 : 0)) {  // R = v - front k S
#pragma unroll
                    for (int a = 0; a < 4; ++a) R[a] = value(a) - front(a) * R[a];
                    split<3>(R[0], R[1], rf[0]);
                }
                if constexpr (g == P::nQ - 1) values(min(c + 1, nc - 1), x_);
            } else if constexpr (x == kT) {  // E = T R, or T^T R
                if constexpr (g == 0) split<3>(R[BWD ? 0 : 2], R[BWD ? 1 : 3], rf[BWD ? 0 : 1]);
                products<3, 3, nt>([&](int k, int i) { return from[3 * k + i]; }, [&](int, int j) { return rf[tb][j]; },
                                   [&](int k) -> f32x4 & { return E[t0 + k]; });
                if constexpr (!BWD && g == 1) {
                    if constexpr (SPLIT == 2) take(given_o, halves_o[w ^ 1], O, 2);
#pragma unroll
                    for (int a = 0; a < NO; ++a) O[a] = (HOLD ? held_o[a] : front(mine_of(a))) * O[a];
                }
                if constexpr (!BWD && g == 0 && NT == 1) decay();
                // the rows of E that the other block does not reach are done
                if constexpr (!BWD && g == 1) {
                    split<3>(wb(0) * E[0], wb(1) * E[1], ef[0]);
                    if constexpr (NT == 3) split<NX>(E[0], E[1], of[0]);
                }
                if constexpr (BWD && g == 1) {
                    split<3>(-front(2) * E[2], -front(3) * E[3], ef[1]);
                    if constexpr (P::late == 0) split<3>(-front(0) * E[0], -front(1) * E[1], ef[0]);
                }
            } else if constexpr (x == kP && !BWD) {  // o = front q S + Q E
                if constexpr (NT == 3 && g == 0) {
                    decay();
                    split<NX>(E[2], E[3], of[1]);
                    split<3>(wb(2) * E[2], wb(3) * E[3], ef[1]);
                    if constexpr (KEEP) put_tokens();  // not held any longer: registers
                }
                constexpr int first = SPLIT == 2 ? g : t0;
                products<NX, NX, NO - first>([&](int k, int i) { return from[NX * k + i]; }, [&](int, int j) { return of[g][j]; },
                                             [&](int k) -> f32x4 & { return O[first + k]; });
                if constexpr (NT == 1 && g == 0) ahead();
                if constexpr (NT == 1 && g == 1) put_rows();
            } else if constexpr (x == kP) {  // Q^T do
                products<3, NT, nt>([&](int k, int i) { return from[3 * k + i]; }, [&](int, int j) { return df[g][j]; },
                                    [&](int k) -> f32x4 & { return O[t0 + k]; });
                split<3>(front(2 * g) * value(2 * g), front(2 * g + 1) * value(2 * g + 1), xf[g]);
                if constexpr (g == 1) values(max(c - 1, 0), x_);
            } else {  // S = whole S + k^T (wb E), or whole S + q^T (front do) - k^T (front E)
                constexpr int b = g * P::GC / (2 * L);
                if constexpr (SPLIT == 2 && x == kQC && g == 0) give(given, halves[w], R, 4);
                products<NT, 3, P::GC>([&](int k, int i) { return from[k * NT + i]; },
                                       [&](int, int j) { return x == kC ? ef[b][j] : xf[b][j]; },
                                       [&](int k) -> f32x4 & { return S[(g * P::GC + k) % (2 * L)]; });
                if constexpr (SPLIT == 2 && x == kQC && g == 0) take(given, halves[w ^ 1], R, 4);
                if constexpr (x == kQC && g == 0) {  // R = Q^T do + wb k G
#pragma unroll
                    for (int a = 0; a < 4; ++a) R[a] = O[a] + wb(a) * R[a];
                    split<3>(R[2], R[3], rf[1]);
                }
                if constexpr (x == kQC && P::late > 0 && g == P::nC - P::late) split<3>(-front(0) * E[0], -front(1) * E[1], ef[0]);
                if constexpr (!BWD && NT == 1) {
                    if constexpr (g == 0) split<3>(wb(2) * E[2], wb(3) * E[3], ef[1]);
                    if constexpr (g == P::nC - 1) {
                        split<NX>(E[0], E[1], of[0]);
                        split<NX>(E[2], E[3], of[1]);
                    }
                }
                if constexpr (x == kC && g == 0) {
                    if constexpr (KEEP && (BWD || NT == 1)) put_tokens();
                    if constexpr (BWD || NT == 3) put_rows();
                }
                if constexpr (x == kC && g == P::nC - 1 && (BWD || NT == 3)) ahead();
            }
        };
        lds_barrier();  // the chunk's operands are there
        bf16x8 f[2][kGroup];
        load(std::integral_constant<int, 0>(), f[0]);
        if constexpr (HOLD) {
#pragma unroll
            for (int a = 0; a < 8; ++a) held[a] = gate(a);
            if constexpr (!BWD) {
                held_o[0] = gate(h);
                held_o[1] = gate(3 - h);
            }
        }
        each<0, P::groups>([&](auto G) __attribute__((always_inline)) {
            constexpr int g = G;
            if constexpr (g + 1 < P::groups) load(std::integral_constant<int, g + 1>(), f[(g + 1) & 1]);
            __builtin_amdgcn_sched_barrier(0);
            run(G, f[g & 1]);
            // a matrix instruction takes the time of four others: three of the vector ALU between two of them
            each<0, 24>([&](auto) __attribute__((always_inline)) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
            });
        });
        if constexpr (P::sets == 1) lds_barrier();  // k is no longer read
    }
    float *last = BWD ? p.dS0 : p.ST;
    if (last) keep(last + head * sstate, S);
}

template <bool BWD, bool KEEP>
const void *pick(int nt, int kb, int nw, bool split) {
    auto of = [&](auto NT, auto KB) -> const void * {
        // an fp32 wave with half of 128 channels that also stores what it keeps has not enough registers for a split
        if constexpr (NT == 3 && KB == 4 && KEEP) {
            if (nw == 2) return reinterpret_cast<const void *>(&delta_chain_kernel<NT, KB, BWD, KEEP, 2, 1>);
        } else {
            if (split) return reinterpret_cast<const void *>(&delta_chain_kernel<NT, KB, BWD, KEEP, 4, 2>);
        }
        return reinterpret_cast<const void *>(&delta_chain_kernel<NT, KB, BWD, KEEP, 4, 1>);
    };
    typedef std::integral_constant<int, 1> one;
    typedef std::integral_constant<int, 2> two;
    typedef std::integral_constant<int, 3> three;
    typedef std::integral_constant<int, 4> four;
    return nt == 1 ? (kb == 2 ? of(one(), two()) : of(one(), four())) : (kb == 2 ? of(three(), two()) : of(three(), four()));
}

// How the chains of a call are launched.
struct Launch {
    int heads;      // value heads of sequences, a multiple of 8, so that the workgroups of one head run on one of the 8 XCDs
                    // (workgroups go round them in turn) and share its operands in that one's cache
    bool split;     // two waves to a tile
    int nw;         // waves of a workgroup that have tiles
    int groups;     // workgroups of a head
    unsigned threads() const { return 64 * (nw + kLoaders); }
};

Launch plan(const DeltaParams &p, bool keep) {
    Launch r;
    r.heads = (int)(((long)p.nseq * p.Hv + 7) / 8 * 8);
    const int nt = p.io_bf16 ? 1 : 3, kb = delta_blocks(p.dk), tiles = delta_col_tiles(p.dv);
    // Two tiles to a workgroup while a compute unit has one such workgroup at most: then the time is that of one chunk after
    // the other.  Their two waves each (16 heads of 1,024 tokens, 128 x 128, bf16, kept: 55 us, with one wave to a tile 61, four tiles to a
    // workgroup 66; 64 heads 70, 72, 75).  With more heads four tiles share what is copied (80 heads 78 us, two to a workgroup 111).
    const bool few = (long)r.heads * ((tiles + 1) / 2) <= 256;
    r.split = few && !(nt == 3 && kb == 4 && keep);  // (64 heads, fp32, kept: split 266 us, not 156)
    r.nw = few && !r.split ? 2 : 4;
    const int per = few ? 2 : 4;
    r.groups = (tiles + per - 1) / per;
    return r;
}

}  // namespace

long delta_chain_threads(const DeltaParams &p) {
    const Launch r = plan(p, false);  // what is kept changes only launches of at most 256 workgroups
    return (long)r.heads * r.groups * r.threads();
}

hipError_t launch_delta_chain(const DeltaParams &p0, bool bwd, hipStream_t s) {
    DeltaParams p = p0;
    const bool keep = p.ckpt != nullptr;
    Launch r = plan(p, keep);
    void *args[] = {&p, &r.heads};
    const int nt = p.io_bf16 ? 1 : 3, kb = delta_blocks(p.dk);
    const void *fn = bwd ? pick<true, true>(nt, kb, r.nw, r.split)
                     : keep ? pick<false, true>(nt, kb, r.nw, r.split) : pick<false, false>(nt, kb, r.nw, r.split);
    return hipLaunchKernel(fn, dim3((unsigned)r.heads * r.groups), dim3(r.threads()), args, 0, s);
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
