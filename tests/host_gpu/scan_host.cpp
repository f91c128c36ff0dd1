// scan_host.cpp -- the gated linear recurrence's entry points and kernels, compiled for the CPU
// from the library's own sources, run once on the case that comes in on stdin, every tensor
// between guard pages (tests/test_scan_host.py).
#include <pthread.h>
#include <stdio.h>
#include <stdlib.h>
#include <sys/mman.h>
#include <ucontext.h>
#include <unistd.h>

#include <atomic>
#include <functional>
#include <thread>
#include <vector>

#include "scan_fwd.hip"

#include "scan_bwd.hip"

#include "scan.hip"

#include "mixer_api.hip"

// the preparation is not part of this program
namespace gdr {
size_t qk_prep_bwd_workspace(const QkParams &) { return 0; }
hipError_t launch_qk_prep(const QkParams &, bool, hipStream_t) { return hipErrorInvalidValue; }
}  // namespace gdr

// what the compiler calls to round an fp32 value to bf16
extern "C" __bf16 __truncsfbf2(float f) {
    const uint16_t h = gdr::f32_to_bf16(f);
    __bf16 b;
    memcpy(&b, &h, 2);
    return b;
}

thread_local uint3 threadIdx, blockIdx;
thread_local dim3 blockDim, gridDim;

// ---------------------------------------------------------------------------
// a workgroup: fibers on the thread that runs it
// ---------------------------------------------------------------------------
struct Group {
    static constexpr int kMost = 512, kStack = 64 << 10;
    ucontext_t lane[kMost], main;
    bool done[kMost];
    char *stacks;
    int n, cur, waiting, turn;            // the barrier: lanes that wait, barriers passed
    int wave_waiting[8], wave_turn[8];
    uint32_t slot[kMost];
    std::function<void()> body;

    Group() {
        stacks = static_cast<char *>(mmap(nullptr, (size_t)kMost * kStack, PROT_READ | PROT_WRITE,
                                          MAP_PRIVATE | MAP_ANONYMOUS | MAP_NORESERVE, -1, 0));
        if (stacks == MAP_FAILED) abort();
    }
    ~Group() { munmap(stacks, (size_t)kMost * kStack); }
    void others() { swapcontext(&lane[cur], &main); }
    void wave_sync() {
        const int w = cur >> 6, t = wave_turn[w];
        if (++wave_waiting[w] == 64) {
            wave_waiting[w] = 0;
            ++wave_turn[w];
        }
        while (wave_turn[w] == t) others();
    }
    void run(int lanes);
};
static thread_local Group *group;

static void enter() {
    group->body();
    group->done[group->cur] = true;
    group->others();
}

void Group::run(int lanes) {
    n = lanes;
    waiting = turn = 0;
    memset(wave_waiting, 0, sizeof(wave_waiting));
    memset(wave_turn, 0, sizeof(wave_turn));
    for (int i = 0; i < n; ++i) {
        done[i] = false;
        getcontext(&lane[i]);
        lane[i].uc_stack.ss_sp = stacks + (size_t)i * kStack;
        lane[i].uc_stack.ss_size = kStack;
        lane[i].uc_link = nullptr;
        makecontext(&lane[i], enter, 0);
    }
    for (int left = n; left > 0;) {
        left = 0;
        for (int i = 0; i < n; ++i) {
            if (done[i]) continue;
            cur = i;
            threadIdx.x = (unsigned)i;
            swapcontext(&main, &lane[i]);
            left += !done[i];
        }
    }
}

void host_barrier() {
    const int t = group->turn;
    if (++group->waiting == group->n) {
        group->waiting = 0;
        ++group->turn;
    }
    while (group->turn == t) group->others();
}

uint32_t host_exchange(uint32_t value, int from) {
    const int me = group->cur;
    group->slot[me] = value;
    group->wave_sync();
    const uint32_t got = group->slot[(me & ~63) + from];
    group->wave_sync();
    return got;
}

bool host_all(bool p) {
    const int me = group->cur;
    group->slot[me] = p;
    group->wave_sync();
    bool all = true;
    for (int i = 0; i < 64; ++i) all &= group->slot[(me & ~63) + i] != 0;
    group->wave_sync();
    return all;
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
static int resident = 16;  // workgroups that run at the same time
static bool skip_first;    // the first block of a pass is never run: the blocks behind it wait in vain

hipError_t hipLaunchKernel(const void *fn, dim3 grid, dim3 block, void **args, size_t, hipStream_t) {
    std::function<void()> body;
    if (fn == reinterpret_cast<const void *>(&gdr::scan_fill_kernel)) {
        body = [=] { gdr::scan_fill_kernel(*static_cast<gdr::u32x4 **>(args[0]), *static_cast<long *>(args[1])); };
    } else if (fn == reinterpret_cast<const void *>(&gdr::scan_copy_kernel)) {
        body = [=] {
            gdr::scan_copy_kernel(*static_cast<const float **>(args[0]), *static_cast<float **>(args[1]), *static_cast<long *>(args[2]));
        };
    } else {
        const gdr::ScanParams p = *static_cast<gdr::ScanParams *>(args[0]);
        if (skip_first && p.nblk > 1) *static_cast<uint32_t *>(p.ws) = 0;
        body = [=] { reinterpret_cast<void (*)(gdr::ScanParams)>(const_cast<void *>(fn))(p); };
    }
    std::atomic<unsigned> next{0};
    std::vector<std::thread> threads;
    for (unsigned t = 0; t < std::min<unsigned>(resident, grid.x); ++t)
        threads.emplace_back([&] {
            Group g;
            group = &g;
            g.body = body;
            gridDim = grid;
            blockDim = block;
            for (unsigned b; (b = next++) < grid.x;) {
                blockIdx.x = b;
                g.run((int)block.x);
            }
        });
    for (std::thread &t : threads) t.join();
    return hipSuccess;
}

// ---------------------------------------------------------------------------
// one case
// ---------------------------------------------------------------------------
// `bytes` of memory between pages that cannot be accessed, at either end of its own pages
static char *guarded(size_t bytes, bool at_end) {
    const size_t page = 4096, own = (bytes + page - 1) / page * page;
    char *p = static_cast<char *>(mmap(nullptr, own + 2 * page, PROT_NONE, MAP_PRIVATE | MAP_ANONYMOUS, -1, 0));
    if (p == MAP_FAILED || (own && mprotect(p + page, own, PROT_READ | PROT_WRITE))) abort();
    memset(p + page, 0x5a, own);
    return at_end ? p + page + own - bytes : p + page;
}

static void *input(size_t bytes, bool at_end) {
    char *p = guarded(bytes, at_end);
    if (fread(p, 1, bytes, stdin) != bytes) abort();
    return p;
}

int main() {
    struct {
        int64_t B, T, H, dv, io, gate, flags, ldx, lda, ldb, beta, n_seq, states, at_end, resident, skip_first;
    } c;
    if (fread(&c, sizeof(c), 1, stdin) != 1) return 2;
    alarm(100);
    resident = (int)c.resident;
    const gdr_desc d = {(int)c.B, (int)c.T, (int)c.H, 1, (int)c.dv, 64, (int)c.io, (int)c.gate, GDR_ALPHA_CHANNEL, 0, (int)c.flags};
    const bool packed = c.n_seq >= 0, e = c.at_end != 0;
    const size_t es = c.io == GDR_BF16 ? 2 : 4, gs = c.gate == GDR_BF16 ? 2 : 4;
    const size_t rows = c.B * c.T, D = c.H * c.dv, n = packed ? c.n_seq : c.B, nblk = (c.T + GDR_SCAN_BLOCK - 1) / GDR_SCAN_BLOCK;
    auto strided = [&](int64_t ld, size_t size) { return rows ? ((rows - 1) * ld + D) * size : 0; };
    const void *x = input(strided(c.ldx, es), e), *alpha = input(strided(c.lda, gs), e);
    const void *beta = c.beta ? input(strided(c.ldb, gs), e) : nullptr;
    const int32_t *off = packed ? static_cast<int32_t *>(input((n + 1) * 4, e)) : nullptr;
    const float *S0 = c.states ? static_cast<float *>(input(n * D * 4, e)) : nullptr;
    const void *dy = input(rows * D * es, e);
    const float *dST = c.states ? static_cast<float *>(input(n * D * 4, e)) : nullptr;
    char *y = guarded(rows * D * es, e), *dx = guarded(rows * D * es, e), *dalpha = guarded(rows * D * gs, e);
    char *dbeta = beta ? guarded(rows * D * gs, e) : nullptr;
    float *ST = reinterpret_cast<float *>(guarded(n * D * 4, e)), *dS0 = reinterpret_cast<float *>(guarded(n * D * 4, e));
    float *ckpt = reinterpret_cast<float *>(guarded(c.B * nblk * D * 4, e));
    const size_t need = gdr_scan_workspace_size(&d);
    char *ws = guarded((need + 15) / 16 * 16, e);
    skip_first = c.skip_first != 0;
    int rc = gdr_scan_fwd(&d, x, c.ldx, alpha, c.lda, beta, c.ldb, off, packed ? (int)n : 0, S0, y, ST, ckpt, ws, need, nullptr);
    if (rc) return 10 - rc;
    skip_first = false;
    rc = gdr_scan_bwd(&d, x, c.ldx, alpha, c.lda, beta, c.ldb, off, packed ? (int)n : 0, S0, ckpt, dy, dST, dx, dalpha, dbeta, dS0,
                      ws, need, nullptr);
    if (rc) return 20 - rc;
    auto output = [](const void *p, size_t bytes) {
        if (p && fwrite(p, 1, bytes, stdout) != bytes) abort();
    };
    output(y, rows * D * es);
    output(ST, n * D * 4);
    output(ckpt, c.B * nblk * D * 4);
    output(dx, rows * D * es);
    output(dalpha, rows * D * gs);
    output(dbeta, rows * D * gs);
    output(dS0, n * D * 4);
    fflush(stdout);
    return 0;
}
