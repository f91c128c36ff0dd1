// delta_api.hip -- the C-ABI entry points of the trainable delta rule and of the block norm (include/gdr.h):
// host-side validation and launches on the caller's stream.
#include <stdint.h>

#include "block_norm.hpp"
#include "checks.hpp"
#include "delta.hpp"
#include "gdr.h"
#include "mixer.hpp"

namespace gdr {
namespace {

int check_delta_desc(const gdr_delta_desc *d) {
    if (!d || d->B < 0 || d->T < 0 || d->Hk < 0 || d->Hv < 0) return GDR_EINVAL;
    if (d->io_dtype != GDR_BF16 && d->io_dtype != GDR_F32) return GDR_EINVAL;
    if (d->gate_dtype != GDR_BF16 && d->gate_dtype != GDR_F32) return GDR_EINVAL;
    if (d->Hk == 0 ? d->Hv != 0 : d->Hv == 0 || d->Hv % d->Hk != 0) return GDR_EINVAL;
    if (d->dk < 8 || d->dk > 128 || (d->dk & 7) || d->dv < 8 || d->dv > 128 || (d->dv & 7)) return GDR_EUNSUPPORTED;
    if ((long long)d->B * d->T > 0x3fffffffLL || d->Hk > 65536 || d->Hv > 65536) return GDR_EUNSUPPORTED;
    return GDR_OK;
}

struct DeltaCall {
    DeltaParams p;
    Span in[6];  // q, k, v, log_gate, beta, seq_off
    long long rows, states;
    size_t es, gs;
    bool empty;  // nothing to compute
};

// Descriptor, sequences, strides: what no pointer is needed for.
int delta_call(const gdr_delta_desc *d, const int32_t *seq_off, int32_t n_seq, DeltaCall &c, bool step = false) {
    const int rc = check_delta_desc(d);
    if (rc) return rc;
    if (n_seq < 0 || (!seq_off && n_seq != 0)) return GDR_EINVAL;
    if (seq_off && d->B != 1) return GDR_EINVAL;
    DeltaParams &p = c.p;
    p = DeltaParams{};
    p.B = d->B;
    p.T = d->T;
    p.Hk = d->Hk;
    p.Hv = d->Hv;
    p.dk = d->dk;
    p.dv = d->dv;
    p.group = d->Hk > 0 ? d->Hv / d->Hk : 1;
    p.io_bf16 = d->io_dtype == GDR_BF16;
    p.gate_bf16 = d->gate_dtype == GDR_BF16;
    p.off = seq_off;
    p.nseq = seq_off ? n_seq : d->B;
    p.chunks = (int)(((long long)d->T + GDR_DELTA_CHUNK - 1) / GDR_DELTA_CHUNK);
    const long long slots = seq_off ? d->T / GDR_DELTA_CHUNK + (long long)n_seq : (long long)d->B * p.chunks;
    if (slots * d->Hv > kMaxThreads / 512) return GDR_EUNSUPPORTED;  // of a launch
    if ((long long)p.nseq * d->Hv > kMaxThreads / 512 - 8) return GDR_EUNSUPPORTED;
    if (!step && delta_chain_threads(p) > kMaxThreads) return GDR_EUNSUPPORTED;
    p.nslot = d->T > 0 ? (int)slots : 0;
    c.rows = (long long)d->B * d->T;
    c.states = (long long)p.nseq * d->Hv * d->dk * d->dv;
    c.es = p.io_bf16 ? 2 : 4;
    c.gs = p.gate_bf16 ? 2 : 4;
    c.empty = p.nseq == 0 || d->Hv == 0;
    p.ldq = d->ldq;
    p.ldk = d->ldk;
    p.ldv = d->ldv;
    p.ldg = d->ldg;
    p.ldb = d->ldb;
    const long long key = (long long)d->Hk * d->dk, value = (long long)d->Hv * d->dv;
    if (!stride_ok(p.ldq, c.rows, key) || !stride_ok(p.ldk, c.rows, key) || !stride_ok(p.ldv, c.rows, value) ||
        !stride_ok(p.ldg, c.rows, d->Hv) || !stride_ok(p.ldb, c.rows, d->Hv))
        return GDR_EINVAL;
    if (key > kMaxRow || value > kMaxRow) return GDR_EUNSUPPORTED;
    // a chunk's rows span less than 2^30 bytes; a step takes rows by themselves
    if (!step && (p.ldq > kMaxRow || p.ldk > kMaxRow || p.ldv > kMaxRow || p.ldg > kMaxRow || p.ldb > kMaxRow)) return GDR_EUNSUPPORTED;
    return GDR_OK;
}

int delta_inputs(DeltaCall &c, const void *q, const void *k, const void *v, const void *g, const void *b) {
    DeltaParams &p = c.p;
    if (c.rows > 0 && !c.empty && (!q || !k || !v || !g || !b)) return GDR_EINVAL;
    if (!aligned_to(q, c.es) || !aligned_to(k, c.es) || !aligned_to(v, c.es) || !aligned_to(g, c.gs) || !aligned_to(b, c.gs))
        return GDR_EINVAL;
    if (!aligned_to(p.off, 4)) return GDR_EINVAL;
    p.q = q;
    p.k = k;
    p.v = v;
    p.g = g;
    p.b = b;
    c.in[0] = {q, extent(c.rows, (long long)p.Hk * p.dk, p.ldq, c.es)};
    c.in[1] = {k, extent(c.rows, (long long)p.Hk * p.dk, p.ldk, c.es)};
    c.in[2] = {v, extent(c.rows, (long long)p.Hv * p.dv, p.ldv, c.es)};
    c.in[3] = {g, extent(c.rows, p.Hv, p.ldg, c.gs)};
    c.in[4] = {b, extent(c.rows, p.Hv, p.ldb, c.gs)};
    c.in[5] = {p.off, p.off ? (size_t)(p.nseq + 1ll) * 4 : 0};
    return GDR_OK;
}

size_t ckpt_bytes(const DeltaParams &p) { return (size_t)p.nslot * p.Hv * delta_tiles(p.dk, p.dv) * 1024; }

int check_norm_desc(const gdr_block_norm_desc *d) {
    if (!d || d->B < 0 || d->T < 0 || d->H < 0) return GDR_EINVAL;
    if (d->io_dtype != GDR_BF16 && d->io_dtype != GDR_F32) return GDR_EINVAL;
    if (d->weight_dtype != GDR_BF16 && d->weight_dtype != GDR_F32) return GDR_EINVAL;
    if (d->norm < GDR_NORM_NONE || d->norm > GDR_NORM_RMS || d->next_norm < GDR_NORM_NONE || d->next_norm > GDR_NORM_RMS)
        return GDR_EINVAL;
    if (d->act < GDR_ACT_LINEAR || d->act > GDR_ACT_SILU) return GDR_EINVAL;
    if (!(d->eps >= 0.f) || d->scale != d->scale || d->res_scale != d->res_scale) return GDR_EINVAL;
    if (d->d < 8 || d->d > kMaxNormWidth || (d->d & 7)) return GDR_EUNSUPPORTED;
    const long long tokens = (long long)d->B * d->T;
    if (tokens > 0x7fffffffLL || (d->H > 0 && tokens > 0x7fffffffLL / d->H)) return GDR_EUNSUPPORTED;
    return GDR_OK;
}

NormParams norm_params(const gdr_block_norm_desc *d) {
    NormParams p{};
    p.rows = (int64_t)d->B * d->T * d->H;
    p.H = d->H;
    p.d = d->d;
    p.io_bf16 = d->io_dtype == GDR_BF16;
    p.w_bf16 = d->weight_dtype == GDR_BF16;
    p.norm = d->norm;
    p.next = d->next_norm != GDR_NORM_NONE;
    p.act = d->act;
    p.kappa = d->norm == GDR_NORM_RMS ? 1.f / (float)d->d : 1.f;
    p.next_kappa = d->next_norm == GDR_NORM_RMS ? 1.f / (float)d->d : 1.f;
    p.eps = d->eps;
    p.scale = d->scale;
    p.res_scale = d->res_scale;
    p.ldx = d->ldx;
    p.ldz = d->ldg;
    p.ldr = d->ldr;
    return p;
}

int norm_inputs(const gdr_block_norm_desc *d, NormParams &p, const void *x, const void *gate, const void *residual, const void *w,
                const void *w_next, Span (&in)[5]) {
    const size_t es = p.io_bf16 ? 2 : 4, ws = p.w_bf16 ? 2 : 4;
    const long long tokens = (long long)d->B * d->T, width = (long long)d->H * d->d;
    if (!stride_ok(p.ldx, tokens, width) || !stride_ok(p.ldz, tokens, width) || !stride_ok(p.ldr, tokens, width)) return GDR_EINVAL;
    if (p.rows > 0 && !x) return GDR_EINVAL;
    if (w_next && !p.next) return GDR_EINVAL;
    if (!aligned_to(x, es) || !aligned_to(gate, es) || !aligned_to(residual, es) || !aligned_to(w, ws) || !aligned_to(w_next, ws))
        return GDR_EINVAL;
    p.x = x;
    p.z = gate;
    p.res = residual;
    p.w = w;
    p.w2 = w_next;
    in[0] = {x, extent(tokens, width, p.ldx, es)};
    in[1] = {gate, extent(tokens, width, p.ldz, es)};
    in[2] = {residual, extent(tokens, width, p.ldr, es)};
    in[3] = {w, ws * d->d};
    in[4] = {w_next, ws * d->d};
    return GDR_OK;
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

size_t gdr_delta_workspace_size(const gdr_delta_desc *d, int32_t n_seq, int32_t backward) {
    DeltaCall c;
    static const int32_t packed = 0;  // only says that the rows are packed
    if (delta_call(d, n_seq > 0 ? &packed : nullptr, n_seq, c) || c.empty || c.p.nslot == 0) return 0;
    return delta_workspace(c.p, backward != 0, nullptr);
}

size_t gdr_delta_ckpt_size(const gdr_delta_desc *d, int32_t n_seq) {
    DeltaCall c;
    static const int32_t packed = 0;
    if (delta_call(d, n_seq > 0 ? &packed : nullptr, n_seq, c) || c.empty) return 0;
    return ckpt_bytes(c.p);
}

int gdr_delta_fwd(const gdr_delta_desc *d, const void *q, const void *k, const void *v, const void *log_gate, const void *beta,
                  const int32_t *seq_off, int32_t n_seq, const float *S0, void *o, float *ST, float *ckpt, void *workspace,
                  size_t workspace_bytes, void *stream) {
    DeltaCall c;
    int rc = delta_call(d, seq_off, n_seq, c);
    if (rc) return rc;
    rc = delta_inputs(c, q, k, v, log_gate, beta);
    if (rc) return rc;
    DeltaParams &p = c.p;
    if (c.rows > 0 && !c.empty && !o) return GDR_EINVAL;
    if (!aligned_to(o, c.es) || !aligned16(S0) || !aligned16(ST) || !aligned16(ckpt)) return GDR_EINVAL;
    const size_t need = c.empty || p.nslot == 0 ? 0 : delta_workspace(p, false, static_cast<char *>(workspace));
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace))) return GDR_EWORKSPACE;
    {
        const size_t nstate = (size_t)c.states * 4;
        const bool resume = ST && ST == S0;
        if (resume && p.off) return GDR_EINVAL;
        Span ins[7];
        for (int i = 0; i < 6; ++i) ins[i] = c.in[i];
        ins[6] = {resume ? nullptr : S0, nstate};
        const Span outs[] = {{o, (size_t)c.rows * p.Hv * p.dv * c.es}, {ST, nstate}, {ckpt, ckpt_bytes(p)},
                             {need ? workspace : nullptr, need}};
        if (!apart(outs, 4, ins, 7)) return GDR_EINVAL;
    }
    if (c.empty) return GDR_OK;
    p.S0 = S0;
    p.o = o;
    p.ST = ST;
    p.ckpt = ckpt;
    return launch_delta_fwd(p, static_cast<hipStream_t>(stream)) == hipSuccess ? GDR_OK : GDR_EHIP;
}

int gdr_delta_bwd(const gdr_delta_desc *d, const void *q, const void *k, const void *v, const void *log_gate, const void *beta,
                  const int32_t *seq_off, int32_t n_seq, const float *ckpt, const void *d_o, const float *dST, void *dq, void *dk,
                  void *dv, void *dlog_gate, void *dbeta, float *dS0, void *workspace, size_t workspace_bytes, void *stream) {
    DeltaCall c;
    int rc = delta_call(d, seq_off, n_seq, c);
    if (rc) return rc;
    rc = delta_inputs(c, q, k, v, log_gate, beta);
    if (rc) return rc;
    DeltaParams &p = c.p;
    if (c.rows > 0 && !c.empty && (!ckpt || !d_o || !dq || !dk || !dv || !dlog_gate || !dbeta)) return GDR_EINVAL;
    if (!aligned_to(d_o, c.es) || !aligned_to(dq, c.es) || !aligned_to(dk, c.es) || !aligned_to(dv, c.es)) return GDR_EINVAL;
    if (!aligned_to(dlog_gate, c.gs) || !aligned_to(dbeta, c.gs)) return GDR_EINVAL;
    if (!aligned16(ckpt) || !aligned16(dST) || !aligned16(dS0)) return GDR_EINVAL;
    const size_t need = c.empty || p.nslot == 0 ? 0 : delta_workspace(p, true, static_cast<char *>(workspace));
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace))) return GDR_EWORKSPACE;
    {
        const size_t nstate = (size_t)c.states * 4, nk = (size_t)c.rows * p.Hk * p.dk * c.es, nv = (size_t)c.rows * p.Hv * p.dv * c.es;
        const size_t ng = (size_t)c.rows * p.Hv * c.gs;
        Span ins[9];
        for (int i = 0; i < 6; ++i) ins[i] = c.in[i];
        ins[6] = {ckpt, ckpt_bytes(p)};
        ins[7] = {d_o, nv};
        ins[8] = {dST, nstate};
        const Span outs[] = {{dq, nk}, {dk, nk}, {dv, nv}, {dlog_gate, ng}, {dbeta, ng}, {dS0, nstate}, {need ? workspace : nullptr, need}};
        if (!apart(outs, 7, ins, 9)) return GDR_EINVAL;
    }
    if (c.empty) return GDR_OK;
    p.ckpt = const_cast<float *>(ckpt);
    p.dout = d_o;
    p.dST = dST;
    p.dq = dq;
    p.dkk = dk;
    p.dvv = dv;
    p.dg = dlog_gate;
    p.db = dbeta;
    p.dS0 = dS0;
    return launch_delta_bwd(p, static_cast<hipStream_t>(stream)) == hipSuccess ? GDR_OK : GDR_EHIP;
}

int gdr_delta_step(const gdr_delta_desc *d, const void *q, const void *k, const void *v, const void *log_gate, const void *beta,
                   float *S, void *o, void *stream) {
    if (!d) return GDR_EINVAL;
    gdr_delta_desc one = *d;  // a step is one token, whatever the descriptor's T
    one.T = 1;
    DeltaCall c;
    int rc = delta_call(&one, nullptr, 0, c, true);
    if (rc) return rc;
    rc = delta_inputs(c, q, k, v, log_gate, beta);
    if (rc) return rc;
    if (c.empty) return GDR_OK;
    if (!S || !o || !aligned16(S) || !aligned_to(o, c.es)) return GDR_EINVAL;
    const Span outs[] = {{S, (size_t)c.states * 4}, {o, (size_t)c.rows * d->Hv * d->dv * c.es}};
    if (!apart(outs, 2, c.in, 5)) return GDR_EINVAL;
    DeltaStepParams p{};
    p.B = d->B;
    p.Hk = d->Hk;
    p.Hv = d->Hv;
    p.dk = d->dk;
    p.dv = d->dv;
    p.group = c.p.group;
    p.io_bf16 = c.p.io_bf16;
    p.gate_bf16 = c.p.gate_bf16;
    p.q = q;
    p.k = k;
    p.v = v;
    p.g = log_gate;
    p.b = beta;
    p.ldq = c.p.ldq;
    p.ldk = c.p.ldk;
    p.ldv = c.p.ldv;
    p.ldg = c.p.ldg;
    p.ldb = c.p.ldb;
    p.S = S;
    p.o = o;
    return launch_delta_step(p, static_cast<hipStream_t>(stream)) == hipSuccess ? GDR_OK : GDR_EHIP;
}

int gdr_block_norm_fwd(const gdr_block_norm_desc *d, const void *x, const void *gate, const void *residual, const void *w,
                       const void *w_next, void *y, void *n, void *stream) {
    int rc = check_norm_desc(d);
    if (rc) return rc;
    NormParams p = norm_params(d);
    Span in[5];
    rc = norm_inputs(d, p, x, gate, residual, w, w_next, in);
    if (rc) return rc;
    if (!p.next && n) return GDR_EINVAL;
    if (p.rows == 0) return GDR_OK;
    if (!y || (p.next && !n)) return GDR_EINVAL;
    const size_t es = p.io_bf16 ? 2 : 4, bytes = (size_t)p.rows * p.d * es;
    if (!aligned_to(y, es) || !aligned_to(n, es)) return GDR_EINVAL;
    // y may be the dense residual: a lane reads its channels of a row before it writes them
    const bool self = y == residual && p.ldr == (int64_t)d->H * d->d;
    const Span outs[] = {{y, bytes}, {n, bytes}};
    if (overlaps(y, bytes, n, bytes)) return GDR_EINVAL;
    for (int i = 0; i < 5; ++i) {
        if (!(i == 2 && self) && overlaps(outs[0].p, outs[0].n, in[i].p, in[i].n)) return GDR_EINVAL;
        if (overlaps(outs[1].p, outs[1].n, in[i].p, in[i].n)) return GDR_EINVAL;
    }
    p.y = y;
    p.n = n;
    return launch_block_norm(p, false, static_cast<hipStream_t>(stream)) == hipSuccess ? GDR_OK : GDR_EHIP;
}

size_t gdr_block_norm_bwd_workspace_size(const gdr_block_norm_desc *d) {
    if (check_norm_desc(d)) return 0;
    return block_norm_workspace(norm_params(d));
}

int gdr_block_norm_bwd(const gdr_block_norm_desc *d, const void *x, const void *gate, const void *residual, const void *w,
                       const void *w_next, const void *dy, const void *dn, void *dx, void *dgate, void *dresidual, float *dw,
                       float *dw_next, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_norm_desc(d);
    if (rc) return rc;
    NormParams p = norm_params(d);
    Span in[5];
    rc = norm_inputs(d, p, x, gate, residual, w, w_next, in);
    if (rc) return rc;
    const size_t es = p.io_bf16 ? 2 : 4, bytes = (size_t)p.rows * p.d * es, wide = (size_t)p.d * 4;
    if ((dw && !w) || (dw_next && !w_next) || !aligned_to(dw, 4) || !aligned_to(dw_next, 4)) return GDR_EINVAL;
    if (!p.next && dn) return GDR_EINVAL;
    if ((dgate && !gate) || (dresidual && !residual)) return GDR_EINVAL;
    if (p.rows > 0) {
        if (!dy || !dx || (p.next && !dn) || (gate && !dgate) || (residual && !dresidual)) return GDR_EINVAL;
        if (!aligned_to(dy, es) || !aligned_to(dn, es) || !aligned_to(dx, es) || !aligned_to(dgate, es) || !aligned_to(dresidual, es))
            return GDR_EINVAL;
    }
    const size_t need = dw || dw_next ? block_norm_workspace(p) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace))) return GDR_EWORKSPACE;
    {
        const Span ins[] = {in[0], in[1], in[2], in[3], in[4], {dy, bytes}, {dn, bytes}};
        const Span outs[] = {{dx, bytes}, {dgate, bytes}, {dresidual, bytes}, {dw, wide}, {dw_next, wide}, {need ? workspace : nullptr, need}};
        if (!apart(outs, 6, ins, 7)) return GDR_EINVAL;
    }
    p.dy = dy;
    p.dn = dn;
    p.dx = dx;
    p.dz = dgate;
    p.dres = dresidual;
    p.dw = dw;
    p.dw2 = dw_next;
    p.partial = static_cast<float *>(workspace);
    return launch_block_norm(p, true, static_cast<hipStream_t>(stream)) == hipSuccess ? GDR_OK : GDR_EHIP;
}

}  // extern "C"
