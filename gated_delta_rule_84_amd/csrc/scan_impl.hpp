// scan_impl.hpp -- gated linear recurrence per channel (include/gdr.h: gdr_scan_fwd, gdr_scan_bwd,
// gdr_scan_step): the mathematics and what its kernels share.  scan_fwd.hip and scan_bwd.hip hold the
// passes over long sequences, scan.hip the single-token step.
//
//     h_t = a_t h_{t-1} + b_t x_t,   y_t = h_t        (per channel, state in fp32)
//
// A token is the affine map h -> a h + u with u = b x; maps compose associatively,
// (A2, U2) o (A1, U1) = (A2 A1, A2 U1 + U2), so a block of tokens is reduced in parallel.
// The backward pass is the same recurrence run from the end.  With G_t the gradient that
// token t hands to t - 1,
//     g_t = dy_t + G_{t+1},  G_t = a_t g_t        (G_{T+1} = dS_T, dS_0 = G_1)
//     dx = b g,  dbeta = g x,  da = g h_{t-1}  (- g x where b = 1 - a)
// and h_{t-1} is formed again inside each block from the state that the forward pass kept
// at the block's border, so no state of a token is stored or read.
//
// Layout: a workgroup of 512 threads takes a block of 256 tokens x 64 channels.  16 lanes hold a
// row of the block (4 channels each) and a lane holds 8 tokens one after the other (a strand),
// all of its inputs in registers between the reduction and the second pass, so every input is
// read once.  The strands' maps are composed over a wave by shuffles, over the 8 waves in shared
// memory and over the blocks of a sequence by the chain below.
//
// Bound by HBM: forward 3 or 4 streams over the tokens for some 25 operations per element,
// backward 5 or 7; where few channels leave few workgroups, by the chain.  Smaller blocks (128
// tokens) or larger ones (512, or 16 tokens per lane), 8 channels per lane and a fixed tile of
// columns per L2 cache were slower or no faster.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdr.h"
#include "gdr_device.hpp"
#include "gdr_mfma.hpp"
#include "mixer.hpp"

namespace gdr {
namespace {

constexpr int kBlk = GDR_SCAN_BLOCK;  // tokens per block
constexpr int kChainHead = 256;       // bytes before the chain's words: the counter of blocks

// How the input factor b is given.
enum Factor { kOne = 0, kGiven = 1, kCoupled = 2 };

// One shape for every pair of types: 16 lanes of 4 channels make rows of 128 bytes of bf16, a whole
// cache line (with 8 lanes, 64 bytes, a bf16 stream reached 3.8 TB/s where it now reaches 5.1), and
// strands of 8 tokens keep 16 loads of a lane in flight.
constexpr int V = 4, L = 8;          // channels per lane, tokens per strand
constexpr int kLR = 16;              // lanes per row
constexpr int kWS = 64 / kLR;        // strands per wave
constexpr int kThreads = kBlk / L * kLR;
constexpr int kWaves = kThreads / 64;
constexpr int CH = kLR * V;          // channels per workgroup, one per lane of the wave that joins the chain

// A range of memory that the hardware checks: loads past its end give 0, stores past it do nothing.
typedef __amdgpu_buffer_rsrc_t Buf;

__device__ __forceinline__ Buf buf(const void *base, int64_t at, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(static_cast<char *>(const_cast<void *>(base)) + at, 0, base ? (int)bytes : 0, 0x00020000);
}

constexpr uint32_t kNowhere = 0x80000000u;  // an offset past every range: they hold at most 2^30 bytes

// V elements of one token, packed as they are stored.
template <bool BF>
struct Pack {
    static constexpr int N = BF ? V / 2 : V, es = BF ? 2 : 4;
    uint32_t w[N];

    __device__ __forceinline__ float get(int v) const {
        if constexpr (BF) return (v & 1) ? __uint_as_float(w[v / 2] & 0xffff0000u) : __uint_as_float(w[v / 2] << 16);
        return __uint_as_float(w[v]);
    }
    // members v and v + 1 (v even)
    __device__ __forceinline__ void set2(int v, float a, float b) {
        if constexpr (BF) {
            w[v / 2] = pk_bf16(a, b);
        } else {
            w[v] = __float_as_uint(a);
            w[v + 1] = __float_as_uint(b);
        }
    }
    // V elements at byte `at`
    __device__ __forceinline__ void load(Buf r, uint32_t at) {
        if constexpr (N == 2) {
            const u32x2 a = __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0);
            w[0] = a[0];
            w[1] = a[1];
        } else {
#pragma unroll
            for (int k = 0; k < N; k += 4) {
                const u32x4 a = __builtin_amdgcn_raw_buffer_load_b128(r, at + 4 * k, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) w[k + i] = a[i];
            }
        }
    }
    __device__ __forceinline__ void store(Buf r, uint32_t at) const {
        if constexpr (N == 2) {
            __builtin_amdgcn_raw_buffer_store_b64((u32x2){w[0], w[1]}, r, at, 0, 0);
        } else {
#pragma unroll
            for (int k = 0; k < N; k += 4)
                __builtin_amdgcn_raw_buffer_store_b128((u32x4){w[k], w[k + 1], w[k + 2], w[k + 3]}, r, at + 4 * k, 0, 0);
        }
    }
    // the first n of the V elements alone
    __device__ __forceinline__ void load(Buf r, uint32_t at, int n) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t o = v < n ? at + v * es : kNowhere;
            if constexpr (BF) {
                const uint32_t h = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, o, 0, 0);
                w[v / 2] = v & 1 ? w[v / 2] | h << 16 : h;
            } else {
                w[v] = __builtin_amdgcn_raw_buffer_load_b32(r, o, 0, 0);
            }
        }
    }
    __device__ __forceinline__ void store(Buf r, uint32_t at, int n) const {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t o = v < n ? at + v * es : kNowhere;
            if constexpr (BF)
                __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(w[v / 2] >> (16 * (v & 1))), r, o, 0, 0);
            else
                __builtin_amdgcn_raw_buffer_store_b32(w[v], r, o, 0, 0);
        }
    }
    // its words where `keep`, else `other`
    __device__ __forceinline__ void choose(bool keep, uint32_t other) {
#pragma unroll
        for (int k = 0; k < N; ++k) w[k] = keep ? w[k] : other;
    }
};

// The fp32 states of all sequences, [n, D]: row i, the lane's channels.  Channels past the row's end
// read what follows it (or 0) and are never stored.
struct States {
    Buf r;
    uint32_t row, ch;
    __device__ __forceinline__ States(const float *base, int n, int D, int ch0)
        : r(buf(base, 0, (uint32_t)n * (uint32_t)D * 4)), row((uint32_t)D * 4), ch((uint32_t)ch0 * 4) {}
    __device__ __forceinline__ void load(int i, float (&f)[V]) const {
        Pack<false> w;
        w.load(r, i * row + ch);
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] = w.get(v);
    }
    __device__ __forceinline__ float load1(int i, int v) const {
        return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, i * row + ch + 4 * v, 0, 0));
    }
    __device__ __forceinline__ void store1(int i, int v, int n, float f) const {
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(f), r, v < n ? i * row + ch + 4 * v : kNowhere, 0, 0);
    }
    __device__ __forceinline__ void store(int i, int n, const float (&f)[V]) const {
#pragma unroll
        for (int v = 0; v < V; ++v) store1(i, v, n, f[v]);
    }
};

// exp(x) and 1 - exp(x), both to 2 units in the last place, by Cody and Waite's two-part reduction, for x in -88 .. 88 (below, 0 and 1;
// above, as at 88).  With n = rint(x / ln 2) and r = x - n ln 2 (ln 2 in two parts), exp(x) = s + s q
// and exp(x) - 1 = (s - 1) + s q for s = 2^n and q = exp(r) - 1, a polynomial on |r| <= 0.35 whose
// first term left out is r^8 / 8! < 2^-26 r.  For x near 0, where 1 - exp(x) would cancel, s = 1 and
// the result is q itself.  n = -127, the least, makes the bit pattern of s that of 0.
__device__ __forceinline__ void exp_both(float x, float &a, float &b) {
    const float y = __builtin_amdgcn_fmed3f(x, -88.f, 88.f);
    const float n = rintf(y * 1.44269504f);
    float r = fmaf(n, -0.693145752f, y);
    r = fmaf(n, -1.42860677e-6f, r);
    float q = fmaf(r, 1.f / 5040, 1.f / 720);
    q = fmaf(r, q, 1.f / 120);
    q = fmaf(r, q, 1.f / 24);
    q = fmaf(r, q, 1.f / 6);
    q = fmaf(r, q, 0.5f);
    q = fmaf(r * r, q, r);
    const float s = __uint_as_float(((uint32_t)(int)n << 23) + 0x3f800000u);
    a = x == x ? fmaf(s, q, s) : x;
    b = x == x ? fmaf(-s, q, 1.f - s) : x;
}

// Decays and input factors of a lane's channels of one token (b is 1 for kOne).
template <int F, bool LOG, bool GB>
__device__ __forceinline__ void gates(const Pack<GB> &al, const Pack<GB> &be, float (&a)[V], float (&b)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        a[v] = al.get(v);
        b[v] = 1.f - a[v];
        if (LOG) exp_both(al.get(v), a[v], b[v]);
        b[v] = F == kGiven ? be.get(v) : (F == kCoupled ? b[v] : 1.f);
    }
}

// Tokens of a strand that are in no sequence become ones that change nothing: a = 1, b x = 0.
template <bool LOG, bool IOB, bool GB, int LB>
__device__ __forceinline__ void leave_out(unsigned in, Pack<IOB> (&x)[L], Pack<GB> (&al)[L], Pack<GB> (&be)[LB]) {
#pragma unroll
    for (int j = 0; j < L; ++j) {
        const bool keep = in >> j & 1;
        x[j].choose(keep, 0);
        be[j % LB].choose(keep, 0);
        al[j].choose(keep, LOG ? 0 : (GB ? 0x3f803f80u : 0x3f800000u));
    }
}

// The rows of a block of one tensor: from the block's first row to the end of the last one that is
// there, so rows past T are past the range, and so is a lane whose channels are past D.
template <bool BF>
struct Rows {
    static constexpr int es = BF ? 2 : 4;
    Buf r;
    uint32_t at, step;
    __device__ __forceinline__ Rows(const void *t, int64_t row, int rows, int64_t ld, int D, int local, int ch)
        : r(buf(t, row * ld * es, ((uint32_t)(rows - 1) * (uint32_t)ld + (uint32_t)D) * es)),
          at(ch < D ? ((uint32_t)local * (uint32_t)ld + (uint32_t)ch) * es : kNowhere), step((uint32_t)ld * es) {}
    // `whole`: each lane has all of its V channels in the row or none, else n of them (element by element:
    // 8 x 1,000 tokens of 1,020 bf16 channels, forward 25.0 us so and 21.4 us whole)
    __device__ __forceinline__ void load(Pack<BF> (&x)[L], bool whole, int n) const {
        if (whole) {
#pragma unroll
            for (int j = 0; j < L; ++j) x[j].load(r, at + j * step);
        } else {
#pragma unroll
            for (int j = 0; j < L; ++j) x[j].load(r, at + j * step, n);
        }
    }
    __device__ __forceinline__ void store(const Pack<BF> (&x)[L], unsigned in, bool whole, int n) const {
        if (whole) {
#pragma unroll
            for (int j = 0; j < L; ++j) x[j].store(r, in >> j & 1 ? at + j * step : kNowhere);
        } else {
#pragma unroll
            for (int j = 0; j < L; ++j) x[j].store(r, at + j * step, in >> j & 1 ? n : 0);
        }
    }
};

// The tokens t0 .. t0 + L - 1 of a strand: bit j of `in` where the token belongs to a sequence,
// of `first` / `last` where it opens / closes one; seq[j] its sequence.  Offsets are read
// with sequence numbers clamped to 0 .. nseq, whatever they hold.
template <bool PACKED>
struct Marks {
    unsigned in = 0, first = 0, last = 0;
    int seq[L];

    __device__ __forceinline__ void find(const ScanParams &p, int t0, unsigned there) {
        if constexpr (PACKED) {
            int lo = 0, hi = p.nseq;  // first sequence that ends after t0
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (p.off[mid + 1] <= t0) lo = mid + 1;
                else hi = mid;
            }
            int i = lo;
#pragma unroll
            for (int j = 0; j < L; ++j) {
                const int t = t0 + j;
                while (i < p.nseq && p.off[i + 1] <= t) ++i;
                const bool ok = i < p.nseq && (there >> j & 1) && p.off[i] <= t;
                seq[j] = ok ? i : 0;
                in |= (unsigned)ok << j;
                first |= (unsigned)(ok && p.off[i] == t) << j;
                last |= (unsigned)(ok && p.off[i + 1] == t + 1) << j;
            }
        } else {
            in = there;
        }
    }
};

// ---------------------------------------------------------------------------
// The chain of blocks: the single-pass scan with decoupled look-back (Merrill and Garland, 2016), with
// affine maps in the place of sums and groups of blocks as a second level.  Every block publishes its composed map as soon as it has it.  The last block
// of each group composes the group's map from them and publishes that, and the state behind
// the group once it is known.  A block takes the state behind the nearest group before it whose state
// is there, applies the maps of the groups in between and then those of its own group's blocks.  What
// is applied to what does not depend on which words were there first, so neither do the results.
// Groups shorten the wait where few channels leave only the chain.  Forward, bf16, log gates, in groups
// of 4 / 6 / 8 blocks: 65,536 tokens of 128 channels 36.6 / 31.2 / 28.7 us, 400,000 of 40 channels
// 142 / 106 / 89 us, against 298 / 298 / 304 us for 65,536 of 4,096, where the data is what counts.
// The backward kernel loses 3 % of its rate on 65,536 x 2,032 with groups of 8 (371 against 358 us),
// nothing with 6.  The packed forward kernel has all of its 128 registers in use with 4 (its fp32 forms with
// beta spill 11 of them, and 16 with log gates as well) and would spill more with larger groups.
// Words are stored and loaded whole with relaxed atomics that all eight L2 caches see; a word is there
// once it is no longer kNone, which no value is stored as, so no order between words matters.
// Blocks are numbered by a counter when they begin: every block before a waiting one is running or
// done, so each wait ends.
constexpr uint32_t kNone = 0xffffffffu;  // what scan_fill_kernel leaves
constexpr uint32_t kCut = 0xfffffffeu;   // in a map's factor: nothing of what enters gets through
constexpr int kGroupFwd = 8, kGroupPacked = 4, kGroupBwd = 6;  // blocks per group (kGroupPacked: forward with offsets)
static_assert(kGroupPacked <= kGroupFwd && kGroupPacked <= kGroupBwd, "scan_workspace takes the smallest");
constexpr int kWindow = 2;               // groups looked back over at a time
// Looks before a wait gives up, a bound that a sound run never meets: a look is a trip past the L2 caches, over
// 100 ns, so half a second at least.  The state is NaN then, and so are the blocks behind.
constexpr int kMaxPolls = 1 << 22;

__device__ __forceinline__ uint32_t word(float f) {
    const uint32_t u = __float_as_uint(f);
    return u >= kCut ? 0x7fc00000u : u;  // two NaN patterns are taken
}

// A composed map of one channel, as published: the factor above, the summand below.
struct Map {
    uint32_t A;
    float U;
    __device__ __forceinline__ float apply(float h) const { return A == kCut ? U : fmaf(__uint_as_float(A), h, U); }
    // this map, then `next`
    __device__ __forceinline__ Map then(const Map &next) const {
        const bool cut = A == kCut || next.A == kCut;
        return {cut ? kCut : word(__uint_as_float(A) * __uint_as_float(next.A)), next.apply(U)};
    }
    __device__ __forceinline__ uint64_t bits() const { return (uint64_t)A << 32 | __float_as_uint(U); }
    static __device__ __forceinline__ Map of(uint64_t w) { return {(uint32_t)(w >> 32), __uint_as_float((uint32_t)w)}; }
};

__device__ __forceinline__ void put(uint64_t *p, uint64_t v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ void put(uint32_t *p, uint32_t v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ uint64_t look(const uint64_t *p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ uint32_t look(const uint32_t *p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// Words of a chain, for one channel: a map per block, a map and a state per group.
__host__ __device__ constexpr int groups_of(int nblk, int group) { return (nblk + group - 1) / group; }
__host__ __device__ constexpr long chain_words(int nblk, int group) { return 2l * nblk + 3l * groups_of(nblk, group); }

template <int GROUP>
struct Chain {
    uint64_t *map, *gmap;
    uint32_t *gstate;
    int nblk;

    // the words of one column (sequence and tile of channels), the lane's channel c
    __device__ __forceinline__ Chain(const ScanParams &p, unsigned column, int c) : nblk(p.nblk) {
        char *ws = static_cast<char *>(p.ws) + kChainHead + column * (chain_words(nblk, GROUP) * CH * 4);
        map = reinterpret_cast<uint64_t *>(ws) + c;
        gmap = map + (long)nblk * CH;
        gstate = reinterpret_cast<uint32_t *>(ws + 8l * (nblk + groups_of(nblk, GROUP)) * CH) + c;
    }
    // The state behind group g - 1 (g > 0; group 0 gives its state without a map).
    __device__ __forceinline__ float group_enters(int g) const {
        for (int poll = 0; poll < kMaxPolls; ++poll) {
            uint32_t h[kWindow];
            uint64_t m[kWindow];
#pragma unroll
            for (int w = 0; w < kWindow; ++w) {
                const int j = g - 1 - w;
                h[w] = kNone;
                m[w] = ~0ull;
                if (j < 0) continue;
                h[w] = look(gstate + (long)j * CH);
                m[w] = look(gmap + (long)j * CH);
            }
            // nearest group whose state is there for every channel, with every map after it
            int from = -1;
            bool maps = true;
#pragma unroll
            for (int w = 0; w < kWindow; ++w) {
                if (from >= 0 || !maps) continue;
                if (__all(h[w] != kNone)) from = w;
                else maps = __all((uint32_t)(m[w] >> 32) != kNone);
            }
            if (from >= 0) {
                float s = 0.f;
#pragma unroll
                for (int w = kWindow - 1; w >= 0; --w) {
                    if (w == from) s = __uint_as_float(h[w]);
                    if (w < from) s = Map::of(m[w]).apply(s);
                }
                return s;
            }
            __builtin_amdgcn_s_sleep(1);
        }
        return __uint_as_float(0x7fc00000u);
    }
    // Joins block k, whose map is `own`, `start` being the state before block 0 (read for k = 0 only):
    // the state that enters the block, and in `out` the one behind it.  Block 0 publishes the state behind
    // it as a map that lets nothing through, so no other block reads S0, which the last block's ST may be:
    // that block begins to store once it has block 0's word, and block 0 has it only from S0.
    __device__ __forceinline__ float join(int k, const Map &block, float start, float &out) const {
        const Map own = k == 0 ? Map{kCut, block.apply(start)} : block;
        const int g = k / GROUP, r = k % GROUP;
        const bool closes = r == GROUP - 1 && k < nblk - 1;  // the last group's state enters nothing
        if (r < GROUP - 1 && k < nblk - 1) put(map + (long)k * CH, own.bits());
        uint64_t m[GROUP - 1];  // of the group's blocks before this one
        bool there = false;
#pragma unroll
        for (int i = 0; i < GROUP - 1; ++i) m[i] = i < r ? look(map + (long)(g * GROUP + i) * CH) : 0;
        for (int poll = 0; !there && poll < kMaxPolls; ++poll) {
            there = true;
#pragma unroll
            for (int i = 0; i < GROUP - 1; ++i) {
                if (__all((uint32_t)(m[i] >> 32) != kNone)) continue;  // only what is missing is looked for again
                m[i] = look(map + (long)(g * GROUP + i) * CH);
                there = false;
            }
        }
        Map all = {0, 0.f};
        if (closes) {
            all = Map::of(m[0]);
#pragma unroll
            for (int i = 1; i < GROUP - 1; ++i) all = all.then(Map::of(m[i]));
            all = all.then(own);
            if (g > 0) put(gmap + (long)g * CH, all.bits());
        }
        float h = g > 0 ? group_enters(g) : start;
        const float behind = all.apply(h);
        if (closes) put(gstate + (long)g * CH, word(behind));
#pragma unroll
        for (int i = 0; i < GROUP - 1; ++i)
            if (i < r) h = Map::of(m[i]).apply(h);
        if (!there) h = __uint_as_float(0x7fc00000u);
        out = closes ? behind : own.apply(h);
        return h;
    }
};

struct Shared {
    float A[kWaves][CH], U[kWaves][CH];  // a wave's composed map, per channel
    int cut[kWaves];                     // it holds a border of sequences
    float in[kWaves][CH];                // the state that enters a wave's strands
};

// Composes the strands of a wave: (A, U) is the lane's own map, afterwards that of the
// wave's strands up to and with its own.  The wave's map goes to shared memory.  REV: the
// strands are taken from the last to the first.  A strand with a border of sequences (`cut`)
// lets nothing of what enters it through: a flag and not A = 0, which would turn an infinity
// of one sequence into a NaN of the next.
template <bool REV, bool PACKED>
__device__ __forceinline__ void compose(Shared &sh, float (&A)[V], float (&U)[V], bool &cut) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, cl = (lane & (kLR - 1)) * V;
    const int strand = REV ? kWS - 1 - lane / kLR : lane / kLR;
#pragma unroll
    for (int s = 1; s < kWS; s <<= 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float a = REV ? __shfl_down(A[v], s * kLR) : __shfl_up(A[v], s * kLR);
            const float u = REV ? __shfl_down(U[v], s * kLR) : __shfl_up(U[v], s * kLR);
            if (strand >= s && !(PACKED && cut)) {
                U[v] = fmaf(A[v], u, U[v]);
                A[v] *= a;
            }
        }
        if (PACKED) {
            const int c = REV ? __shfl_down((int)cut, s * kLR) : __shfl_up((int)cut, s * kLR);
            if (strand >= s) cut = cut || c;
        }
    }
    if (strand == kWS - 1) {
        if (PACKED) sh.cut[wave] = cut;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            sh.A[wave][cl + v] = A[v];
            sh.U[wave][cl + v] = U[v];
        }
    }
}

// One lane per channel: the composed map of the workgroup's waves, in the order of the strands.
template <bool REV, bool PACKED>
__device__ __forceinline__ Map block_map(const Shared &sh, int waves, int c) {
    float a = 1.f, u = 0.f;
    bool cut = false;
    for (int i = 0; i < waves; ++i) {
        const int w = REV ? waves - 1 - i : i;
        if (PACKED && sh.cut[w]) {
            cut = true;
            u = sh.U[w][c];
        } else {
            u = fmaf(sh.A[w][c], u, sh.U[w][c]);
            a *= sh.A[w][c];
        }
    }
    return {cut ? kCut : word(a), u};
}

// One lane per channel: the state that enters each wave when h enters the block.
template <bool REV, bool PACKED>
__device__ __forceinline__ void wave_states(Shared &sh, int waves, int c, float h) {
    for (int i = 0; i < waves; ++i) {
        const int w = REV ? waves - 1 - i : i;
        sh.in[w][c] = h;
        h = PACKED && sh.cut[w] ? sh.U[w][c] : fmaf(sh.A[w][c], h, sh.U[w][c]);
    }
}

// The state that enters the lane's strand.
template <bool REV, bool PACKED>
__device__ __forceinline__ void strand_states(const Shared &sh, const float (&A)[V], const float (&U)[V], bool cut, float (&h)[V]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, cl = (lane & (kLR - 1)) * V;
    const int strand = REV ? kWS - 1 - lane / kLR : lane / kLR;
    const int before = PACKED ? (REV ? __shfl_down((int)cut, kLR) : __shfl_up((int)cut, kLR)) : 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float c = sh.in[wave][cl + v];
        const float a = REV ? __shfl_down(A[v], kLR) : __shfl_up(A[v], kLR);
        const float u = REV ? __shfl_down(U[v], kLR) : __shfl_up(U[v], kLR);
        h[v] = strand ? (PACKED && before ? u : fmaf(a, c, u)) : c;
    }
}

// This workgroup's place: blocks in the order of the recurrence, all channels of one block
// before the next (neighbours read neighbouring memory, and a block's predecessors began long
// before it).  Never past the last place, whatever the counter holds.
__device__ __forceinline__ unsigned place(const ScanParams &p, int &ticket) {
    if (p.nblk == 1) return blockIdx.x;
    if (threadIdx.x == 0) ticket = (int)(atomicAdd(static_cast<uint32_t *>(p.ws), 1u) + 1u);  // starts at kNone
    __syncthreads();
    return min((unsigned)__builtin_amdgcn_readfirstlane(ticket), gridDim.x - 1);  // one value for the wave, held as one
}

// K::get<IOB, GB, F, LOG, PACKED>() is a kernel; the one of a call.
template <class K, bool IOB, bool GB, int F>
const void *pick_rest(const ScanParams &p) {
    if (p.log_gate) return p.off ? K::template get<IOB, GB, F, true, true>() : K::template get<IOB, GB, F, true, false>();
    return p.off ? K::template get<IOB, GB, F, false, true>() : K::template get<IOB, GB, F, false, false>();
}

template <class K, bool IOB, bool GB>
const void *pick_factor(const ScanParams &p) {
    if (p.beta) return pick_rest<K, IOB, GB, kGiven>(p);
    return p.coupled ? pick_rest<K, IOB, GB, kCoupled>(p) : pick_rest<K, IOB, GB, kOne>(p);
}

template <class K>
const void *pick(const ScanParams &p) {
    if (p.io_bf16) return p.gate_bf16 ? pick_factor<K, true, true>(p) : pick_factor<K, true, false>(p);
    return p.gate_bf16 ? pick_factor<K, false, true>(p) : pick_factor<K, false, false>(p);
}

// Columns of a call (sequences times tiles of channels) and the bytes of their chains.
inline long columns_of(const ScanParams &p) { return (long)p.B * ((p.D + CH - 1) / CH); }
inline long chain_bytes(const ScanParams &p, int group) {
    return p.nblk <= 1 ? 0 : kChainHead + columns_of(p) * chain_words(p.nblk, group) * CH * 4;
}

// Waves per workgroup: as many as a call of few tokens has strands for.
inline int waves_of(const ScanParams &p) {
    const int strands = ((p.T < kBlk ? p.T : kBlk) + L - 1) / L;
    return (strands + kWS - 1) / kWS;
}

// Every word of the chain to kNone (a kernel, so that a captured graph replays it): 2.2 us for one
// sequence of few channels, 2.8 us for 4 x 16 blocks of 2,048 channels, 6.5 us for 256 of 4,096.
__global__ void __launch_bounds__(256) scan_fill_kernel(u32x4 *ws, long n) {
    const long i = (long)blockIdx.x * 256 + threadIdx.x;
    if (i < n) ws[i] = (u32x4){kNone, kNone, kNone, kNone};
}

// Clears the chain's words and launches the blocks.
template <class K>
hipError_t launch_blocks(const ScanParams &p, hipStream_t s) {
    const long blocks = columns_of(p) * p.nblk;  // fits: the host has checked the threads
    if (p.nblk > 1) {
        u32x4 *ws = static_cast<u32x4 *>(p.ws);
        long n = chain_bytes(p, K::group(p)) / 16;
        void *args[] = {&ws, &n};
        const hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(&scan_fill_kernel), dim3((unsigned)((n + 255) / 256)),
                                             dim3(256), args, 0, s);
        if (e != hipSuccess) return e;
    }
    ScanParams q = p;
    void *args[] = {&q};
    return hipLaunchKernel(pick<K>(p), dim3((unsigned)blocks), dim3(64 * waves_of(p)), args, 0, s);
}

}  // namespace
}  // namespace gdr
