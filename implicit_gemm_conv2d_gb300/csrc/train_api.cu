// train_api.cu -- the C ABI declared in include/conv_train.h: argument checks (on the host,
// before anything is enqueued) and dispatch to the operators' launchers.
#include <cmath>
#include <cstdint>

#include "train_internal.h"

using namespace igc;

namespace {

constexpr int64_t kMax32 = (int64_t(1) << 31) - 1;

bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int gn_params(const conv_gn_desc_t* d, GnParams& p)
{
    if (!d) return CONV_ERR_NULL;
    if (d->B < 0 || d->C < 1 || d->P < 1 || d->G < 1 || d->C % d->G != 0 || d->act < CONV_ACT_NONE ||
        d->act > CONV_ACT_GELU || (d->layout != CONV_LAYOUT_NCHW && d->layout != CONV_LAYOUT_NHWC) ||
        (d->dtype != CONV_F32 && d->dtype != CONV_BF16) || !std::isfinite(d->eps) || d->eps < 0.f)
        return CONV_ERR_DESC;
    // (B: the kernels step over samples in 32 bits, by B / 128 or some hundred thousand at most)
    if (int64_t(d->C) * d->P > kMax32 - (1 << 20) || int64_t(d->B) * d->G > kMax32 || d->B > kMax32 - (1 << 25))
        return CONV_ERR_UNSUPPORTED;
    p.B = d->B; p.C = d->C; p.P = d->P; p.G = d->G;
    p.Cg = d->C / d->G;
    p.act = d->act;
    p.layout = d->layout;
    p.M = int64_t(p.Cg) * p.P;
    p.N = int64_t(p.C) * p.P;
    p.eps = d->eps;
    p.m = float(p.M);
    p.inv_m = float(1.0 / double(p.M));
    return CONV_OK;
}

int embed_check(const conv_embed_desc_t* d)
{
    if (!d) return CONV_ERR_NULL;
    if (d->T < 0 || d->V < 1 || d->D < 1 || (d->index_dtype != CONV_INDEX_I32 && d->index_dtype != CONV_INDEX_I64) ||
        (d->dtype != CONV_F32 && d->dtype != CONV_BF16) || !std::isfinite(d->scale))
        return CONV_ERR_DESC;
    if (d->T > kMax32 - (1 << 20) || d->D > (1 << 24)) return CONV_ERR_UNSUPPORTED;
    return CONV_OK;
}

int ln_check(const conv_ln_desc_t* d)
{
    if (!d) return CONV_ERR_NULL;
    if (d->N < 0 || d->D < 1 || (d->rms != 0 && d->rms != 1) || (d->dtype != CONV_F32 && d->dtype != CONV_BF16) ||
        !std::isfinite(d->eps) || d->eps < 0.f)
        return CONV_ERR_DESC;
    if (d->N > kMax32 || d->D >= 1 << 30) return CONV_ERR_UNSUPPORTED;
    return CONV_OK;
}

// The last element's offset is one that 64 bits hold in bytes.
bool rows_near(const conv_rows_t& r, int64_t B, int64_t T, int64_t D)
{
    const __int128 top = __int128(B > 0 ? B - 1 : 0) * r.batch + __int128(T > 0 ? T - 1 : 0) * r.step + D;
    return top < __int128(1) << 60;
}

// An output's rows do not overlap, whichever of the two dimensions is the outer one (rows_near holds).
bool rows_apart(const conv_rows_t& r, int64_t B, int64_t T, int64_t D)
{
    if (B <= 1 || T <= 1) return (B <= 1 || T < 1 || r.batch >= D) && (T <= 1 || B < 1 || r.step >= D);
    if (r.step < D || r.batch < D) return false;
    return r.batch >= (T - 1) * r.step + D || r.step >= (B - 1) * r.batch + D;
}

int scan_check(const conv_scan_desc_t* d, bool bwd)
{
    if (!d) return CONV_ERR_NULL;
    if (d->B < 0 || d->T < 0 || d->D < 1 || (d->dtype != CONV_F32 && d->dtype != CONV_BF16)) return CONV_ERR_DESC;
    const conv_rows_t* rows[] = {&d->x, &d->gate, &d->h, &d->dh, &d->dx, &d->dgate};
    const int used = bwd ? 6 : 3;
    for (int i = 0; i < used; ++i)
        if (rows[i]->batch < 0 || rows[i]->step < 0) return CONV_ERR_DESC;
    for (int i = 0; i < used; ++i)
        if (!rows_near(*rows[i], d->B, d->T, d->D)) return CONV_ERR_UNSUPPORTED;
    for (int i = bwd ? 4 : 2; i < used; ++i)
        if (!rows_apart(*rows[i], d->B, d->T, d->D)) return CONV_ERR_DESC;
    const int64_t most = kMax32 - (1 << 20);
    if (d->B > most || d->T > most || d->D > most || int64_t(d->B) * d->D >= int64_t(1) << 37) return CONV_ERR_UNSUPPORTED;
    return CONV_OK;
}

int distill_check(const conv_distill_desc_t* d)
{
    if (!d) return CONV_ERR_NULL;
    if (d->N < 0 || d->V < 1 || d->K < 1 || d->ld < d->V || (d->dtype != CONV_F32 && d->dtype != CONV_BF16) ||
        (d->teacher_dtype != CONV_F32 && d->teacher_dtype != CONV_BF16) ||
        (d->index_dtype != CONV_INDEX_I32 && d->index_dtype != CONV_INDEX_I64) || 
        !(d->temperature >= 0x1p-60f && d->temperature <= 0x1p60f))  // its square and 1 / it are normal numbers
        return CONV_ERR_DESC;
    if (d->N >= 1 << 27 || d->V >= 1 << 30 || d->K > 1024 || d->ld >= int64_t(1) << 32) return CONV_ERR_UNSUPPORTED;
    return CONV_OK;
}

// `clip`: out is checked too.
int grads_check(const conv_grad_t* g, int32_t count, bool clip)
{
    if (count < 0) return CONV_ERR_DESC;
    if (count > (1 << 20)) return CONV_ERR_UNSUPPORTED;
    if (count > 0 && !g) return CONV_ERR_NULL;
    for (int32_t i = 0; i < count; ++i) {
        if (g[i].n < 0 || (g[i].dtype != CONV_F32 && g[i].dtype != CONV_BF16)) return CONV_ERR_DESC;
        if (g[i].n >= int64_t(1) << 40) return CONV_ERR_UNSUPPORTED;
        if (g[i].n == 0) continue;
        const size_t a = g[i].dtype == CONV_F32 ? 4 : 2;
        if (!g[i].grad || (clip && !g[i].out)) return CONV_ERR_NULL;
        if (!aligned_to(g[i].grad, a) || (clip && !aligned_to(g[i].out, a))) return CONV_ERR_ALIGN;
    }
    return CONV_OK;
}

int grads_run(const conv_grad_t* g, int32_t count, bool clip, float max_norm, float* norm, void* ws, size_t ws_bytes,
              conv_stream_t stream)
{
    int rc = grads_check(g, count, clip);
    if (rc != CONV_OK) return rc;
    if (clip && (!std::isfinite(max_norm) || max_norm < 0.f)) return CONV_ERR_DESC;
    if (!norm) return CONV_ERR_NULL;
    if (!aligned_to(norm, 4) || (ws && !aligned16(ws))) return CONV_ERR_ALIGN;
    DevInfo d;
    if ((rc = device_info(d)) != CONV_OK) return rc;
    const size_t need = grad_workspace(g, count, d);
    if (need > 0 && (!ws || ws_bytes < need)) return CONV_ERR_WORKSPACE;
    return cuda_status(run_grad_norm(g, count, clip, max_norm, d, norm, ws, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

size_t conv_gn_fwd_workspace_size(const conv_gn_desc_t* desc)
{
    GnParams p;
    DevInfo d;
    if (gn_params(desc, p) != CONV_OK || device_info(d) != CONV_OK) return 0;
    return gn_fwd_workspace(p, desc->dtype, d);
}

int conv_gn_fwd(const conv_gn_desc_t* desc, const void* x, const void* gamma, const void* beta, void* y, float* mean,
                float* rstd, void* workspace, size_t workspace_bytes, conv_stream_t stream)
{
    GnParams p;
    int rc = gn_params(desc, p);
    if (rc != CONV_OK) return rc;
    if (p.B == 0) return CONV_OK;
    if (!x || !y || (!mean) != (!rstd)) return CONV_ERR_NULL;
    if (!aligned16(x) || !aligned16(y) || !aligned16(gamma) || !aligned16(beta) || !aligned16(mean) ||
        !aligned16(rstd) || !aligned16(workspace))
        return CONV_ERR_ALIGN;
    DevInfo d;
    if ((rc = device_info(d)) != CONV_OK) return rc;
    const size_t need = gn_fwd_workspace(p, desc->dtype, d);
    if (need > 0 && (!workspace || workspace_bytes < need)) return CONV_ERR_WORKSPACE;
    return cuda_status(run_gn_fwd(p, desc->dtype, d, x, gamma, beta, y, mean, rstd, workspace,
                                  reinterpret_cast<cudaStream_t>(stream)));
}

size_t conv_gn_bwd_workspace_size(const conv_gn_desc_t* desc)
{
    GnParams p;
    DevInfo d;
    if (gn_params(desc, p) != CONV_OK || device_info(d) != CONV_OK) return 0;
    return gn_bwd_workspace(p, desc->dtype, d);
}

int conv_gn_bwd(const conv_gn_desc_t* desc, const void* x, const void* dy, const void* gamma, const void* beta,
                const float* mean, const float* rstd, void* dx, void* dgamma, void* dbeta, void* workspace,
                size_t workspace_bytes, conv_stream_t stream)
{
    GnParams p;
    int rc = gn_params(desc, p);
    if (rc != CONV_OK) return rc;
    if ((!dgamma) != (!dbeta)) return CONV_ERR_NULL;
    if (p.B > 0 && (!x || !dy || !mean || !rstd || !dx)) return CONV_ERR_NULL;
    if (!aligned16(dgamma) || !aligned16(dbeta) || !aligned16(workspace) ||
        (p.B > 0 && (!aligned16(x) || !aligned16(dy) || !aligned16(gamma) || !aligned16(beta) || !aligned16(mean) ||
                     !aligned16(rstd) || !aligned16(dx))))
        return CONV_ERR_ALIGN;
    DevInfo d;
    if ((rc = device_info(d)) != CONV_OK) return rc;
    const size_t need = gn_bwd_workspace(p, desc->dtype, d);
    if (need > 0 && (!workspace || workspace_bytes < need)) return CONV_ERR_WORKSPACE;
    return cuda_status(run_gn_bwd(p, desc->dtype, d, x, dy, gamma, beta, mean, rstd, dx, dgamma, dbeta, workspace,
                                  reinterpret_cast<cudaStream_t>(stream)));
}

int conv_embed_fwd(const conv_embed_desc_t* desc, const void* idx, const void* table, void* y, conv_stream_t stream)
{
    int rc = embed_check(desc);
    if (rc != CONV_OK) return rc;
    if (desc->T == 0) return CONV_OK;
    if (!idx || !table || !y) return CONV_ERR_NULL;
    if (!aligned16(idx) || !aligned16(table) || !aligned16(y)) return CONV_ERR_ALIGN;
    DevInfo d;
    if ((rc = device_info(d)) != CONV_OK) return rc;
    return cuda_status(run_embed_fwd(*desc, d, idx, table, y, reinterpret_cast<cudaStream_t>(stream)));
}

size_t conv_embed_bwd_workspace_size(const conv_embed_desc_t* desc)
{
    DevInfo d;
    if (embed_check(desc) != CONV_OK || device_info(d) != CONV_OK) return 0;
    return embed_bwd_workspace(*desc, d);
}

int conv_embed_bwd(const conv_embed_desc_t* desc, const void* idx, const void* dy, void* dtable, void* workspace,
                   size_t workspace_bytes, conv_stream_t stream)
{
    int rc = embed_check(desc);
    if (rc != CONV_OK) return rc;
    if (!dtable || (desc->T > 0 && (!idx || !dy))) return CONV_ERR_NULL;
    if (!aligned16(dtable) || !aligned16(workspace) || (desc->T > 0 && (!aligned16(idx) || !aligned16(dy))))
        return CONV_ERR_ALIGN;
    DevInfo d;
    if ((rc = device_info(d)) != CONV_OK) return rc;
    const size_t need = embed_bwd_workspace(*desc, d);
    if (need > 0 && (!workspace || workspace_bytes < need)) return CONV_ERR_WORKSPACE;
    return cuda_status(run_embed_bwd(*desc, d, idx, dy, dtable, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

int conv_ln_fwd(const conv_ln_desc_t* desc, const void* x, const void* residual, const void* gamma, const void* beta,
                void* y, void* total, float* mean, float* rstd, conv_stream_t stream)
{
    int rc = ln_check(desc);
    if (rc != CONV_OK) return rc;
    if (desc->rms && (beta || mean)) return CONV_ERR_DESC;
    if (desc->N == 0) return CONV_OK;
    if (!x || !y || (!residual) != (!total) || (!desc->rms && (!mean) != (!rstd))) return CONV_ERR_NULL;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(gamma) || !aligned16(beta) || !aligned16(y) ||
        !aligned16(total) || !aligned16(mean) || !aligned16(rstd))
        return CONV_ERR_ALIGN;
    if (y == total) return CONV_ERR_DESC;
    DevInfo d;
    if ((rc = device_info(d)) != CONV_OK) return rc;
    return cuda_status(run_ln_fwd(*desc, d, x, residual, gamma, beta, y, total, mean, rstd,
                                  reinterpret_cast<cudaStream_t>(stream)));
}

size_t conv_ln_bwd_workspace_size(const conv_ln_desc_t* desc)
{
    DevInfo d;
    if (ln_check(desc) != CONV_OK || device_info(d) != CONV_OK) return 0;
    return ln_bwd_workspace(*desc, d);
}

int conv_ln_bwd(const conv_ln_desc_t* desc, const void* x, const void* dy, const void* gamma, const float* mean,
                const float* rstd, const void* dtotal, void* dx, void* dgamma, void* dbeta, void* workspace,
                size_t workspace_bytes, conv_stream_t stream)
{
    int rc = ln_check(desc);
    if (rc != CONV_OK) return rc;
    if (desc->rms && (mean || dbeta)) return CONV_ERR_DESC;
    if (!desc->rms && (!dgamma) != (!dbeta)) return CONV_ERR_NULL;
    if (desc->N > 0 && (!x || !dy || !rstd || !dx || (!desc->rms && !mean))) return CONV_ERR_NULL;
    if (!aligned16(dgamma) || !aligned16(dbeta) || !aligned16(workspace) ||
        (desc->N > 0 && (!aligned16(x) || !aligned16(dy) || !aligned16(gamma) || !aligned16(mean) || !aligned16(rstd) ||
                         !aligned16(dtotal) || !aligned16(dx))))
        return CONV_ERR_ALIGN;
    if (desc->N > 0 && dx == x) return CONV_ERR_DESC;
    DevInfo d;
    if ((rc = device_info(d)) != CONV_OK) return rc;
    const size_t need = ln_bwd_workspace(*desc, d);
    if (need > 0 && (!workspace || workspace_bytes < need)) return CONV_ERR_WORKSPACE;
    return cuda_status(run_ln_bwd(*desc, d, x, dy, gamma, mean, rstd, dtotal, dx, dgamma, dbeta, workspace,
                                  reinterpret_cast<cudaStream_t>(stream)));
}

size_t conv_scan_fwd_workspace_size(const conv_scan_desc_t* desc)
{
    DevInfo d;
    if (scan_check(desc, false) != CONV_OK || device_info(d) != CONV_OK) return 0;
    return scan_workspace(*desc, d, false);
}

size_t conv_scan_bwd_workspace_size(const conv_scan_desc_t* desc)
{
    DevInfo d;
    if (scan_check(desc, true) != CONV_OK || device_info(d) != CONV_OK) return 0;
    return scan_workspace(*desc, d, true);
}

int conv_scan_fwd(const conv_scan_desc_t* desc, const void* x, const void* gate, const float* h0, const uint8_t* reset,
                  const int32_t* lengths, void* h, float* last, void* workspace, size_t workspace_bytes,
                  conv_stream_t stream)
{
    int rc = scan_check(desc, false);
    if (rc != CONV_OK) return rc;
    if (desc->B == 0) return CONV_OK;
    if (desc->T > 0 && (!x || !gate || !h)) return CONV_ERR_NULL;
    const size_t a = desc->dtype == CONV_F32 ? 4 : 2;
    if (!aligned_to(x, a) || !aligned_to(gate, a) || !aligned_to(h, a) || !aligned_to(h0, 4) || !aligned_to(last, 4) ||
        !aligned_to(lengths, 4) || !aligned16(workspace))
        return CONV_ERR_ALIGN;
    if (desc->T > 0 && (h == x || h == gate)) return CONV_ERR_DESC;
    DevInfo d;
    if ((rc = device_info(d)) != CONV_OK) return rc;
    const size_t need = scan_workspace(*desc, d, false);
    if (need > 0 && (!workspace || workspace_bytes < need)) return CONV_ERR_WORKSPACE;
    return cuda_status(run_scan_fwd(*desc, d, x, gate, h0, reset, lengths, h, last, workspace,
                                    reinterpret_cast<cudaStream_t>(stream)));
}

int conv_scan_bwd(const conv_scan_desc_t* desc, const void* x, const void* gate, const void* h, const void* dh,
                  const float* h0, const float* dlast, const uint8_t* reset, const int32_t* lengths, void* dx,
                  void* dgate, float* dh0, void* workspace, size_t workspace_bytes, conv_stream_t stream)
{
    int rc = scan_check(desc, true);
    if (rc != CONV_OK) return rc;
    if (desc->B == 0) return CONV_OK;
    if (desc->T > 0 && (!x || !gate || !h || !dh || !dx || !dgate)) return CONV_ERR_NULL;
    const size_t a = desc->dtype == CONV_F32 ? 4 : 2;
    if (!aligned_to(x, a) || !aligned_to(gate, a) || !aligned_to(h, a) || !aligned_to(dh, a) || !aligned_to(dx, a) ||
        !aligned_to(dgate, a) || !aligned_to(h0, 4) || !aligned_to(dlast, 4) || !aligned_to(dh0, 4) ||
        !aligned_to(lengths, 4) || !aligned16(workspace))
        return CONV_ERR_ALIGN;
    const void* inputs[] = {x, gate, h, dh};
    for (const void* in : inputs)
        if (desc->T > 0 && (dx == in || dgate == in || dx == dgate)) return CONV_ERR_DESC;
    DevInfo d;
    if ((rc = device_info(d)) != CONV_OK) return rc;
    const size_t need = scan_workspace(*desc, d, true);
    if (need > 0 && (!workspace || workspace_bytes < need)) return CONV_ERR_WORKSPACE;
    return cuda_status(run_scan_bwd(*desc, d, x, gate, h, dh, h0, dlast, reset, lengths, dx, dgate, dh0, workspace,
                                    reinterpret_cast<cudaStream_t>(stream)));
}

int conv_distill_fwd(const conv_distill_desc_t* desc, const void* z, const void* ids, const void* teacher, float* loss,
                     float* zmax, float* zlog, conv_stream_t stream)
{
    int rc = distill_check(desc);
    if (rc != CONV_OK) return rc;
    if (desc->N == 0) return CONV_OK;
    if (!z || !ids || !teacher || !loss || !zmax || !zlog) return CONV_ERR_NULL;
    if (!aligned16(z) || !aligned16(ids) || !aligned16(teacher) || !aligned16(loss) || !aligned16(zmax) ||
        !aligned16(zlog))
        return CONV_ERR_ALIGN;
    DevInfo d;
    if ((rc = device_info(d)) != CONV_OK) return rc;
    return cuda_status(
        run_distill_fwd(*desc, d, z, ids, teacher, loss, zmax, zlog, reinterpret_cast<cudaStream_t>(stream)));
}

int conv_distill_bwd(const conv_distill_desc_t* desc, const void* z, const void* ids, const void* teacher,
                     const float* zmax, const float* zlog, const float* weight, float scale, void* dz,
                     conv_stream_t stream)
{
    int rc = distill_check(desc);
    if (rc != CONV_OK) return rc;
    if (!std::isfinite(scale)) return CONV_ERR_DESC;
    if (desc->N == 0) return CONV_OK;
    if (!z || !ids || !teacher || !zmax || !zlog || !dz) return CONV_ERR_NULL;
    if (!aligned16(z) || !aligned16(ids) || !aligned16(teacher) || !aligned16(zmax) || !aligned16(zlog) ||
        !aligned16(weight) || !aligned16(dz))
        return CONV_ERR_ALIGN;
    DevInfo d;
    if ((rc = device_info(d)) != CONV_OK) return rc;
    return cuda_status(run_distill_bwd(*desc, d, z, ids, teacher, zmax, zlog, weight, scale, dz,
                                       reinterpret_cast<cudaStream_t>(stream)));
}

int conv_distill_grad(const conv_distill_desc_t* desc, const void* z, const void* ids, const void* teacher,
                      const float* weight, float scale, float* loss, void* dz, conv_stream_t stream)
{
    int rc = distill_check(desc);
    if (rc != CONV_OK) return rc;
    if (!std::isfinite(scale)) return CONV_ERR_DESC;
    if (desc->N == 0) return CONV_OK;
    if (!z || !ids || !teacher || !loss || !dz) return CONV_ERR_NULL;
    if (!aligned16(z) || !aligned16(ids) || !aligned16(teacher) || !aligned16(loss) || !aligned16(weight) ||
        !aligned16(dz))
        return CONV_ERR_ALIGN;
    DevInfo d;
    if ((rc = device_info(d)) != CONV_OK) return rc;
    return cuda_status(
        run_distill_grad(*desc, d, z, ids, teacher, weight, scale, loss, dz, reinterpret_cast<cudaStream_t>(stream)));
}

size_t conv_grad_norm_workspace_size(const conv_grad_t* grads, int32_t count)
{
    DevInfo d;
    if (grads_check(grads, count, false) != CONV_OK || device_info(d) != CONV_OK) return 0;
    return grad_workspace(grads, count, d);
}

int conv_grad_norm(const conv_grad_t* grads, int32_t count, float* norm, void* workspace, size_t workspace_bytes,
                   conv_stream_t stream)
{
    return grads_run(grads, count, false, 0.f, norm, workspace, workspace_bytes, stream);
}

int conv_grad_clip(const conv_grad_t* grads, int32_t count, float max_norm, float* norm, void* workspace,
                   size_t workspace_bytes, conv_stream_t stream)
{
    return grads_run(grads, count, true, max_norm, norm, workspace, workspace_bytes, stream);
}

}  // extern "C"
