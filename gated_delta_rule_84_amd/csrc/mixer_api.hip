// mixer_api.hip -- the C-ABI entry points of the query / key preparation and of the gated linear
// recurrence (include/gdr.h): host-side validation and launches on the caller's stream.
#include <stdint.h>

#include "checks.hpp"
#include "gdr.h"
#include "mixer.hpp"

namespace gdr {
namespace {

int check_qk_desc(const gdr_qk_desc *d) {
    if (!d || d->B < 0 || d->T < 0 || d->Hq < 0 || d->Hk < 0) return GDR_EINVAL;
    if (d->io_dtype != GDR_BF16 && d->io_dtype != GDR_F32) return GDR_EINVAL;
    if (d->weight_dtype != GDR_BF16 && d->weight_dtype != GDR_F32) return GDR_EINVAL;
    if (d->norm < GDR_NORM_NONE || d->norm > GDR_NORM_RMS) return GDR_EINVAL;
    if (d->rot_layout != GDR_ROT_HALF && d->rot_layout != GDR_ROT_INTERLEAVED) return GDR_EINVAL;
    if (!(d->eps >= 0.f) || !(d->q_scale == d->q_scale) || !(d->rot_scale == d->rot_scale)) return GDR_EINVAL;
    if (d->rot_dim < 0 || (d->rot_dim & 1) || d->rot_dim > d->d) return GDR_EINVAL;
    if (d->d < 8 || d->d > 256 || (d->d & 7)) return GDR_EUNSUPPORTED;
    // a token's number fits 31 bits; rows of heads are counted in 64
    if ((long long)d->B * d->T > 0x3fffffffLL || d->Hq > 65536 || d->Hk > 65536) return GDR_EUNSUPPORTED;
    return GDR_OK;
}

QkParams qk_params(const gdr_qk_desc *d) {
    QkParams p{};
    p.tokens = (int64_t)d->B * d->T;
    p.T = d->T;
    p.d = d->d;
    p.rot = d->rot_dim;
    p.io_bf16 = d->io_dtype == GDR_BF16;
    p.w_bf16 = d->weight_dtype == GDR_BF16;
    p.norm = d->norm;
    p.half_layout = d->rot_layout == GDR_ROT_HALF;
    p.kappa = d->norm == GDR_NORM_NONE ? 0.f : d->norm == GDR_NORM_L2 ? 1.f : 1.f / (float)d->d;
    p.eps = d->eps;
    p.rot_scale = d->rot_scale;
    p.q.H = d->Hq;
    p.k.H = d->Hk;
    p.q.ld = d->ldq;
    p.k.ld = d->ldk;
    p.q.scale = d->q_scale;
    p.k.scale = 1.f;
    return p;
}

// The checks that the forward and the backward pass share; fills the inputs.
int qk_inputs(const gdr_qk_desc *d, QkParams &p, const void *q, const void *k, const void *wq, const void *wk,
              const int32_t *positions, const double *inv_freq) {
    const size_t es = p.io_bf16 ? 2 : 4, wsz = p.w_bf16 ? 2 : 4;
    if (!stride_ok(p.q.ld, p.tokens, (long long)d->Hq * d->d) || !stride_ok(p.k.ld, p.tokens, (long long)d->Hk * d->d))
        return GDR_EINVAL;
    if (d->norm == GDR_NORM_NONE && (wq || wk)) return GDR_EINVAL;
    if (p.tokens > 0 && ((d->Hq > 0 && !q) || (d->Hk > 0 && !k))) return GDR_EINVAL;
    if (p.tokens > 0 && d->rot_dim > 0 && !inv_freq) return GDR_EINVAL;
    if (!aligned_to(q, es) || !aligned_to(k, es) || !aligned_to(wq, wsz) || !aligned_to(wk, wsz)) return GDR_EINVAL;
    if (!aligned_to(positions, 4) || !aligned_to(inv_freq, 8)) return GDR_EINVAL;
    p.q.x = q;
    p.k.x = k;
    p.q.w = wq;
    p.k.w = wk;
    p.pos = positions;
    p.inv_freq = inv_freq;
    return GDR_OK;
}

int check_scan_desc(const gdr_desc *d) {
    if (!d || d->B < 0 || d->T < 0 || d->H < 0) return GDR_EINVAL;
    if (d->io_dtype != GDR_BF16 && d->io_dtype != GDR_F32) return GDR_EINVAL;
    if (d->gate_dtype != GDR_BF16 && d->gate_dtype != GDR_F32) return GDR_EINVAL;
    if (d->alpha_mode != GDR_ALPHA_SCALAR && d->alpha_mode != GDR_ALPHA_CHANNEL) return GDR_EINVAL;
    if (d->flags & ~(GDR_FLAG_LOG_GATE | GDR_FLAG_COUPLED)) return GDR_EINVAL;
    if (d->dv < 1) return GDR_EINVAL;
    if (d->alpha_mode != GDR_ALPHA_CHANNEL) return GDR_EUNSUPPORTED;
    if ((long long)d->H * d->dv > kMaxRow || (long long)d->B * d->T > 0x3fffffffLL) return GDR_EUNSUPPORTED;
    if ((int64_t)d->B * d->H * d->dv * 4 > kMaxStates) return GDR_EUNSUPPORTED;
    return GDR_OK;
}

ScanParams scan_params(const gdr_desc *d) {
    ScanParams p{};
    p.B = d->B;
    p.T = d->T;
    p.D = d->H * d->dv;
    p.io_bf16 = d->io_dtype == GDR_BF16;
    p.gate_bf16 = d->gate_dtype == GDR_BF16;
    p.log_gate = (d->flags & GDR_FLAG_LOG_GATE) != 0;
    p.coupled = (d->flags & GDR_FLAG_COUPLED) != 0;
    p.nblk = (int)(((long long)d->T + GDR_SCAN_BLOCK - 1) / GDR_SCAN_BLOCK);
    return p;
}

// The checks of x, alpha and beta, whose rows are at most `most` elements apart; fills them and their byte extents.
int scan_inputs(ScanParams &p, long long rows, int64_t most, const void *x, int64_t ldx, const void *alpha, int64_t lda,
                const void *beta, int64_t ldb, Span (&in)[3]) {
    const size_t es = p.io_bf16 ? 2 : 4, gs = p.gate_bf16 ? 2 : 4;
    if (!stride_ok(ldx, rows, p.D) || !stride_ok(lda, rows, p.D) || !stride_ok(ldb, rows, p.D)) return GDR_EINVAL;
    if (ldx > most || lda > most || ldb > most) return GDR_EUNSUPPORTED;
    if (p.coupled && beta) return GDR_EINVAL;
    if (rows > 0 && p.D > 0 && (!x || !alpha)) return GDR_EINVAL;
    if (!aligned_to(x, es) || !aligned_to(alpha, gs) || !aligned_to(beta, gs)) return GDR_EINVAL;
    p.x = x;
    p.alpha = alpha;
    p.beta = beta;
    p.ldx = ldx;
    p.lda = lda;
    p.ldb = ldb;
    in[0] = {x, extent(rows, p.D, ldx, es)};
    in[1] = {alpha, extent(rows, p.D, lda, gs)};
    in[2] = {beta, extent(rows, p.D, ldb, gs)};
    return GDR_OK;
}

int scan_sequences(ScanParams &p, const int32_t *seq_off, int32_t n_seq) {
    if (!seq_off) return n_seq == 0 ? GDR_OK : GDR_EINVAL;
    if (n_seq < 0 || !aligned_to(seq_off, 4)) return GDR_EINVAL;
    if (p.B != 1) return GDR_EINVAL;
    if ((int64_t)n_seq * p.D * 4 > kMaxStates) return GDR_EUNSUPPORTED;
    p.off = seq_off;
    p.nseq = n_seq;
    return GDR_OK;
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

int gdr_qk_prep_fwd(const gdr_qk_desc *d, const void *q, const void *k, const void *wq, const void *wk,
                    const int32_t *positions, const double *inv_freq, void *q_out, void *k_out, void *stream) {
    int rc = check_qk_desc(d);
    if (rc) return rc;
    QkParams p = qk_params(d);
    rc = qk_inputs(d, p, q, k, wq, wk, positions, inv_freq);
    if (rc) return rc;
    if (p.tokens == 0) return GDR_OK;
    const size_t es = p.io_bf16 ? 2 : 4, wsz = (p.w_bf16 ? 2 : 4) * (size_t)d->d;
    if ((d->Hq > 0 && !q_out) || (d->Hk > 0 && !k_out)) return GDR_EINVAL;
    if (!aligned_to(q_out, es) || !aligned_to(k_out, es)) return GDR_EINVAL;
    {
        const long long wq_ = (long long)d->Hq * d->d, wk_ = (long long)d->Hk * d->d;
        // an output may be its own dense input: every row is read before it is written
        const bool self_q = q_out == q && p.q.ld == wq_, self_k = k_out == k && p.k.ld == wk_;
        const Span outs[] = {{q_out, p.tokens * wq_ * es}, {k_out, p.tokens * wk_ * es}};
        const Span in_q = {q, extent(p.tokens, wq_, p.q.ld, es)}, in_k = {k, extent(p.tokens, wk_, p.k.ld, es)};
        const Span ins[] = {{wq, wsz}, {wk, wsz}, {positions, (size_t)p.tokens * 4}, {inv_freq, (size_t)(d->rot_dim / 2) * 8}};
        if (!apart(outs, 2, ins, 4)) return GDR_EINVAL;
        if (!self_q && overlaps(outs[0].p, outs[0].n, in_q.p, in_q.n)) return GDR_EINVAL;
        if (!self_k && overlaps(outs[1].p, outs[1].n, in_k.p, in_k.n)) return GDR_EINVAL;
        if (overlaps(outs[0].p, outs[0].n, in_k.p, in_k.n) || overlaps(outs[1].p, outs[1].n, in_q.p, in_q.n)) return GDR_EINVAL;
    }
    p.q.out = q_out;
    p.k.out = k_out;
    return launch_qk_prep(p, false, static_cast<hipStream_t>(stream)) == hipSuccess ? GDR_OK : GDR_EHIP;
}

size_t gdr_qk_prep_bwd_workspace_size(const gdr_qk_desc *d) {
    if (check_qk_desc(d) || d->norm == GDR_NORM_NONE) return 0;
    return qk_prep_bwd_workspace(qk_params(d));
}

int gdr_qk_prep_bwd(const gdr_qk_desc *d, const void *q, const void *k, const void *wq, const void *wk,
                    const int32_t *positions, const double *inv_freq, const void *dq_out, const void *dk_out, void *dq,
                    void *dk, float *dwq, float *dwk, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_qk_desc(d);
    if (rc) return rc;
    QkParams p = qk_params(d);
    rc = qk_inputs(d, p, q, k, wq, wk, positions, inv_freq);
    if (rc) return rc;
    if ((dwq && !wq) || (dwk && !wk) || !aligned_to(dwq, 4) || !aligned_to(dwk, 4)) return GDR_EINVAL;
    const size_t es = p.io_bf16 ? 2 : 4, wsz = (p.w_bf16 ? 2 : 4) * (size_t)d->d, dsz = (size_t)d->d * 4;
    const long long wq_ = (long long)d->Hq * d->d, wk_ = (long long)d->Hk * d->d;
    const size_t nq = p.tokens * wq_ * es, nk = p.tokens * wk_ * es;
    if (p.tokens > 0) {
        if ((d->Hq > 0 && (!dq_out || !dq)) || (d->Hk > 0 && (!dk_out || !dk))) return GDR_EINVAL;
        if (!aligned_to(dq_out, es) || !aligned_to(dk_out, es) || !aligned_to(dq, es) || !aligned_to(dk, es)) return GDR_EINVAL;
    }
    const bool sums = dwq || dwk;
    const size_t need = sums ? qk_prep_bwd_workspace(p) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace))) return GDR_EWORKSPACE;
    {
        const Span outs[] = {{dq, nq}, {dk, nk}, {dwq, dsz}, {dwk, dsz}, {need ? workspace : nullptr, need}};
        const Span ins[] = {{q, extent(p.tokens, wq_, p.q.ld, es)}, {k, extent(p.tokens, wk_, p.k.ld, es)}, {wq, wsz}, {wk, wsz},
                            {positions, (size_t)p.tokens * 4}, {inv_freq, (size_t)(d->rot_dim / 2) * 8}};
        if (!apart(outs, 5, ins, 6)) return GDR_EINVAL;
        const Span gq = {dq_out, nq}, gk = {dk_out, nk};  // a gradient may be overwritten by its own result
        for (int i = 0; i < 5; ++i) {
            if (!(i == 0 && dq == dq_out) && overlaps(outs[i].p, outs[i].n, gq.p, gq.n)) return GDR_EINVAL;
            if (!(i == 1 && dk == dk_out) && overlaps(outs[i].p, outs[i].n, gk.p, gk.n)) return GDR_EINVAL;
        }
    }
    p.q.g = dq_out;
    p.k.g = dk_out;
    p.q.out = dq;
    p.k.out = dk;
    p.q.dw = dwq;
    p.k.dw = dwk;
    p.partial = static_cast<float *>(workspace);
    return launch_qk_prep(p, true, static_cast<hipStream_t>(stream)) == hipSuccess ? GDR_OK : GDR_EHIP;
}

size_t gdr_scan_workspace_size(const gdr_desc *d) {
    if (check_scan_desc(d)) return 0;
    return scan_workspace(scan_params(d));
}

int gdr_scan_fwd(const gdr_desc *d, const void *x, int64_t ldx, const void *alpha, int64_t lda, const void *beta, int64_t ldb,
                 const int32_t *seq_off, int32_t n_seq, const float *S0, void *y, float *ST, float *ckpt, void *workspace,
                 size_t workspace_bytes, void *stream) {
    int rc = check_scan_desc(d);
    if (rc) return rc;
    ScanParams p = scan_params(d);
    const long long rows = (long long)d->B * d->T;
    Span ins[5];
    Span in3[3];
    rc = scan_inputs(p, rows, kMaxRow, x, ldx, alpha, lda, beta, ldb, in3);
    if (rc) return rc;
    rc = scan_sequences(p, seq_off, n_seq);
    if (rc) return rc;
    const size_t es = p.io_bf16 ? 2 : 4;
    const long long ns = p.off ? p.nseq : p.B;
    if (rows > 0 && p.D > 0 && !y) return GDR_EINVAL;
    if (!aligned_to(y, es) || !aligned_to(S0, 4) || !aligned_to(ST, 4) || !aligned_to(ckpt, 4)) return GDR_EINVAL;
    const size_t need = scan_workspace(p);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace))) return GDR_EWORKSPACE;
    {
        const size_t nstate = (size_t)ns * p.D * 4;
        const bool resume = ST && ST == S0;
        if (resume && p.off && rows > 0) return GDR_EINVAL;
        for (int i = 0; i < 3; ++i) ins[i] = in3[i];
        ins[3] = {resume ? nullptr : S0, nstate};
        ins[4] = {seq_off, (size_t)(n_seq + 1ll) * 4};
        const Span outs[] = {{y, (size_t)rows * p.D * es}, {ST, nstate}, {ckpt, (size_t)p.B * p.nblk * p.D * 4},
                             {need ? workspace : nullptr, need}};
        if (!apart(outs, 4, ins, 5)) return GDR_EINVAL;
    }
    if (p.D == 0 || ns == 0) return GDR_OK;
    if (scan_threads(p) > kMaxThreads) return GDR_EUNSUPPORTED;
    p.S0 = S0;
    p.y = y;
    p.ST = ST;
    p.ckpt = ckpt;
    p.ws = workspace;
    return launch_scan_fwd(p, static_cast<hipStream_t>(stream)) == hipSuccess ? GDR_OK : GDR_EHIP;
}

int gdr_scan_bwd(const gdr_desc *d, const void *x, int64_t ldx, const void *alpha, int64_t lda, const void *beta, int64_t ldb,
                 const int32_t *seq_off, int32_t n_seq, const float *S0, const float *ckpt, const void *dy, const float *dST,
                 void *dx, void *dalpha, void *dbeta, float *dS0, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_scan_desc(d);
    if (rc) return rc;
    ScanParams p = scan_params(d);
    const long long rows = (long long)d->B * d->T;
    Span in3[3];
    rc = scan_inputs(p, rows, kMaxRow, x, ldx, alpha, lda, beta, ldb, in3);
    if (rc) return rc;
    rc = scan_sequences(p, seq_off, n_seq);
    if (rc) return rc;
    const size_t es = p.io_bf16 ? 2 : 4, gs = p.gate_bf16 ? 2 : 4;
    const long long ns = p.off ? p.nseq : p.B;
    if ((dbeta != nullptr) != (beta != nullptr) && rows > 0 && p.D > 0) return GDR_EINVAL;
    if (rows > 0 && p.D > 0 && (!dy || !dx || !dalpha)) return GDR_EINVAL;
    if (p.nblk > 1 && p.B > 0 && p.D > 0 && !ckpt) return GDR_EINVAL;
    if (!aligned_to(dy, es) || !aligned_to(dx, es) || !aligned_to(dalpha, gs) || !aligned_to(dbeta, gs)) return GDR_EINVAL;
    if (!aligned_to(S0, 4) || !aligned_to(ckpt, 4) || !aligned_to(dST, 4) || !aligned_to(dS0, 4)) return GDR_EINVAL;
    const size_t need = scan_workspace(p);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace))) return GDR_EWORKSPACE;
    {
        const size_t nstate = (size_t)ns * p.D * 4, nio = (size_t)rows * p.D * es, ng = (size_t)rows * p.D * gs;
        const Span ins[] = {in3[0], in3[1], in3[2], {S0, nstate}, {ckpt, (size_t)p.B * p.nblk * p.D * 4}, {dy, nio}, {dST, nstate},
                            {seq_off, (size_t)(n_seq + 1ll) * 4}};
        const Span outs[] = {{dx, nio}, {dalpha, ng}, {dbeta, ng}, {dS0, nstate}, {need ? workspace : nullptr, need}};
        if (!apart(outs, 5, ins, 8)) return GDR_EINVAL;
    }
    if (p.D == 0 || ns == 0) return GDR_OK;
    if (scan_threads(p) > kMaxThreads) return GDR_EUNSUPPORTED;
    p.S0 = S0;
    p.ckpt = const_cast<float *>(ckpt);
    p.dy = dy;
    p.dST = dST;
    p.dx = dx;
    p.dalpha = dalpha;
    p.dbeta = dbeta;
    p.dS0 = dS0;
    p.ws = workspace;
    return launch_scan_bwd(p, static_cast<hipStream_t>(stream)) == hipSuccess ? GDR_OK : GDR_EHIP;
}

int gdr_scan_step(const gdr_desc *d, const void *x, int64_t ldx, const void *alpha, int64_t lda, const void *beta, int64_t ldb,
                  float *S, void *y, void *stream) {
    if (!d) return GDR_EINVAL;
    gdr_desc one = *d;  // a step is one token, whatever the descriptor's T
    one.T = 1;
    int rc = check_scan_desc(&one);
    if (rc) return rc;
    ScanParams p = scan_params(&one);
    Span ins[3];
    // 64-bit addresses, no block of rows: any stride
    rc = scan_inputs(p, p.B, INT64_MAX, x, ldx, alpha, lda, beta, ldb, ins);
    if (rc) return rc;
    if (p.B == 0 || p.D == 0) return GDR_OK;
    if (!S || !y) return GDR_EINVAL;
    if (!aligned_to(S, 4) || !aligned_to(y, p.io_bf16 ? 2 : 4)) return GDR_EINVAL;
    const Span outs[] = {{S, (size_t)p.B * p.D * 4}, {y, (size_t)p.B * p.D * (p.io_bf16 ? 2 : 4)}};
    if (!apart(outs, 2, ins, 3)) return GDR_EINVAL;
    p.ST = S;
    p.y = y;
    return launch_scan_step(p, static_cast<hipStream_t>(stream)) == hipSuccess ? GDR_OK : GDR_EHIP;
}

}  // extern "C"
