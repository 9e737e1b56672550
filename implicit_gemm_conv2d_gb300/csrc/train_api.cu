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
