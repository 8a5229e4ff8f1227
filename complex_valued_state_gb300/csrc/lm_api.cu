// C ABI entry points of the gated delta rule, of linear attention and of the norms:
// argument validation on the host, workspace handling, and the launches.  See
// include/cssd.h for the contract.

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/cssd.h"
#include "api_checks.h"
#include "cssd_internal.h"

namespace {

using cssd::aligned;
using cssd::check_all_device;
using cssd::stream_device;

constexpr int64_t kMaxInt = 2147483647;

bool supported_type(int t) { return t == CSSD_BF16 || t == CSSD_F16 || t == CSSD_F32; }
bool supported_width(int64_t n) { return n >= 16 && n <= 128 && n % 16 == 0; }

// a * b <= most, for positive values (no overflow).
bool product_fits(int64_t a, int64_t b, int64_t most) { return a <= most / b; }

int check_delta_dims(const cssd_delta_dims* d, int dtype, bool need_seq) {
    if (!d) return CSSD_ERR_NULL;
    if (d->batch <= 0 || d->nheads <= 0 || d->kheads <= 0 || d->dstate <= 0 || d->headdim <= 0) return CSSD_ERR_DIMS;
    if (need_seq && d->seqlen <= 0) return CSSD_ERR_DIMS;
    if (!supported_type(dtype) || !supported_width(d->dstate) || !supported_width(d->headdim)) return CSSD_ERR_UNSUPPORTED;
    if (d->nheads % d->kheads) return CSSD_ERR_DIMS;
    // the kernels index (batch, head, state slice) and (batch, head, chunk) in
    // 32 bits: a step takes up to four slices of a state, a sequence in fp32 one of
    // 16 columns each and its gradients that for two scans in one launch
    const int64_t slices = need_seq && d->headdim / 8 > 4 ? d->headdim / 8 : 4;
    if (d->batch > kMaxInt || d->nheads > kMaxInt || !product_fits(d->batch, d->nheads, kMaxInt / slices)) return CSSD_ERR_DIMS;
    if (need_seq) {
        if (d->seqlen > kMaxInt - 64) return CSSD_ERR_DIMS;
        if (!product_fits(d->batch * d->nheads, (d->seqlen + 63) / 64, kMaxInt)) return CSSD_ERR_DIMS;
    }
    return CSSD_OK;
}

cssd::DeltaArgs delta_args(const cssd_delta_dims* d, int dtype) {
    cssd::DeltaArgs a{};
    a.Bz = d->batch;
    a.T = d->seqlen;
    a.H = d->nheads;
    a.KH = d->kheads;
    a.N = d->dstate;
    a.P = d->headdim;
    a.dtype = dtype;
    return a;
}

// The caller's workspace, or one allocated on the stream (freed by the
// destructor on the same stream).
struct Workspace {
    void* p;
    bool own = false;
    cudaStream_t stream;
    int status = CSSD_OK;
    Workspace(void* given, size_t need, cudaStream_t s) : p(given), stream(s) {
        if (given || !need) return;
        if (cudaMallocAsync(&p, need, s) != cudaSuccess) {
            cudaGetLastError();
            status = CSSD_ERR_WORKSPACE;
            return;
        }
        own = true;
    }
    ~Workspace() {
        if (own) cudaFreeAsync(p, stream);
    }
    Workspace(const Workspace&) = delete;
    Workspace& operator=(const Workspace&) = delete;
};

int status_of(cudaError_t e) {
    if (e == cudaSuccess) return CSSD_OK;
    cudaGetLastError();
    return CSSD_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t cssd_delta_workspace_bytes(const cssd_delta_dims* d, int dtype) {
    if (check_delta_dims(d, dtype, true) != CSSD_OK) return 0;
    return cssd::delta_workspace_bytes(delta_args(d, dtype));
}

size_t cssd_delta_backward_workspace_bytes(const cssd_delta_dims* d, int dtype) {
    if (check_delta_dims(d, dtype, true) != CSSD_OK) return 0;
    return cssd::delta_backward_workspace_bytes(delta_args(d, dtype));
}

int cssd_delta_forward(const cssd_delta_dims* d, int dtype, const void* q, const void* k, const void* v, const float* g,
                       const float* beta, float scale, const float* h0, const int32_t* lens, void* o, float* h_final,
                       void* workspace, size_t workspace_bytes, cssd_stream_t stream_) {
    int s = check_delta_dims(d, dtype, true);
    if (s != CSSD_OK) return s;
    if (!q || !k || !v || !g || !beta || !o) return CSSD_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(h0, 16) ||
        !aligned(h_final, 16) || !aligned(workspace, 16) || !aligned(g, 4) || !aligned(beta, 4) || !aligned(lens, 4))
        return CSSD_ERR_ALIGN;
    cssd::DeltaArgs a = delta_args(d, dtype);
    const size_t need = cssd::delta_workspace_bytes(a);
    if (workspace && workspace_bytes < need) return CSSD_ERR_WORKSPACE;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    int dev = 0;
    if ((s = stream_device(stream, &dev)) != CSSD_OK) return s;
    if ((s = check_all_device(dev, q, k, v, (const void*)g, (const void*)beta, (const void*)h0, (const void*)lens,
                              (const void*)o, (const void*)h_final, (const void*)workspace)) != CSSD_OK)
        return s;
    Workspace ws(workspace, need, stream);
    if (ws.status != CSSD_OK) return ws.status;
    a.scale = scale;
    a.q = q;
    a.k = k;
    a.v = v;
    a.g = g;
    a.beta = beta;
    a.h0 = h0;
    a.lens = lens;
    a.o = o;
    a.h_final = h_final;
    return status_of(cssd::launch_delta_forward(a, ws.p, stream));
}

int cssd_delta_backward(const cssd_delta_dims* d, int dtype, const void* q, const void* k, const void* v, const float* g,
                        const float* beta, float scale, const float* h0, const int32_t* lens, const void* dout,
                        const float* dh_final, void* gq, void* gk, void* gv, float* gg, float* gbeta, float* gh0,
                        void* workspace, size_t workspace_bytes, cssd_stream_t stream_) {
    int s = check_delta_dims(d, dtype, true);
    if (s != CSSD_OK) return s;
    if (!q || !k || !v || !g || !beta || !dout || !gq || !gk || !gv || !gg || !gbeta) return CSSD_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(dout, 16) || !aligned(h0, 16) ||
        !aligned(dh_final, 16) || !aligned(gq, 16) || !aligned(gk, 16) || !aligned(gv, 16) || !aligned(gh0, 16) ||
        !aligned(workspace, 16) || !aligned(g, 4) || !aligned(beta, 4) || !aligned(lens, 4) || !aligned(gg, 4) ||
        !aligned(gbeta, 4))
        return CSSD_ERR_ALIGN;
    cssd::DeltaArgs a = delta_args(d, dtype);
    const size_t need = cssd::delta_backward_workspace_bytes(a);
    if (workspace && workspace_bytes < need) return CSSD_ERR_WORKSPACE;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    int dev = 0;
    if ((s = stream_device(stream, &dev)) != CSSD_OK) return s;
    if ((s = check_all_device(dev, q, k, v, (const void*)g, (const void*)beta, (const void*)h0, (const void*)lens, dout,
                              (const void*)dh_final, (const void*)gq, (const void*)gk, (const void*)gv, (const void*)gg,
                              (const void*)gbeta, (const void*)gh0, (const void*)workspace)) != CSSD_OK)
        return s;
    Workspace ws(workspace, need, stream);
    if (ws.status != CSSD_OK) return ws.status;
    a.scale = scale;
    a.q = q;
    a.k = k;
    a.v = v;
    a.g = g;
    a.beta = beta;
    a.h0 = h0;
    a.lens = lens;
    a.dout = dout;
    a.dh_final = dh_final;
    a.gq = gq;
    a.gk = gk;
    a.gv = gv;
    a.gg = gg;
    a.gbeta = gbeta;
    a.gh0 = gh0;
    return status_of(cssd::launch_delta_backward(a, ws.p, stream));
}

int cssd_delta_step(const cssd_delta_dims* d, int dtype, float* h, int64_t nslots, const int32_t* slots, const void* q,
                    const void* k, const void* v, const float* g, const float* beta, float scale, void* o,
                    cssd_stream_t stream_) {
    int s = check_delta_dims(d, dtype, false);
    if (s != CSSD_OK) return s;
    if (nslots <= 0 || (!slots && nslots < d->batch)) return CSSD_ERR_DIMS;
    if (!h || !q || !k || !v || !g || !beta || !o) return CSSD_ERR_NULL;
    if (!aligned(h, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(g, 4) ||
        !aligned(beta, 4) || !aligned(slots, 4))
        return CSSD_ERR_ALIGN;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    int dev = 0;
    if ((s = stream_device(stream, &dev)) != CSSD_OK) return s;
    if ((s = check_all_device(dev, (const void*)h, (const void*)slots, q, k, v, (const void*)g, (const void*)beta,
                              (const void*)o)) != CSSD_OK)
        return s;
    cssd::DeltaStepArgs a{};
    a.Bz = d->batch;
    a.H = d->nheads;
    a.KH = d->kheads;
    a.N = d->dstate;
    a.P = d->headdim;
    a.nslots = nslots;
    a.dtype = dtype;
    a.scale = scale;
    a.h = h;
    a.slots = slots;
    a.q = q;
    a.k = k;
    a.v = v;
    a.g = g;
    a.beta = beta;
    a.o = o;
    return status_of(cssd::launch_delta_step(a, stream));
}

static int check_norm(int64_t rows, int64_t width, int xtype, int wtype) {
    if (rows <= 0 || width <= 0) return CSSD_ERR_DIMS;
    if (rows > kMaxInt || width > (1 << 24)) return CSSD_ERR_DIMS;
    if (!supported_type(xtype) || (wtype != xtype && wtype != CSSD_F32)) return CSSD_ERR_UNSUPPORTED;
    return CSSD_OK;
}

int cssd_layernorm(int64_t rows, int64_t width, int xtype, int wtype, const void* x, const void* weight,
                   const void* bias, float eps, void* y, float* mean, float* rstd, cssd_stream_t stream_) {
    int s = check_norm(rows, width, xtype, wtype);
    if (s != CSSD_OK) return s;
    if (!(eps >= 0.f)) return CSSD_ERR_DIMS;
    if (!x || !y) return CSSD_ERR_NULL;
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(weight, 16) || !aligned(bias, 16) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return CSSD_ERR_ALIGN;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    int dev = 0;
    if ((s = stream_device(stream, &dev)) != CSSD_OK) return s;
    if ((s = check_all_device(dev, x, weight, bias, (const void*)y, (const void*)mean, (const void*)rstd)) != CSSD_OK)
        return s;
    cssd::NormArgs a{};
    a.rows = rows;
    a.width = width;
    a.xtype = xtype;
    a.wtype = wtype;
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.eps = eps;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    return status_of(cssd::launch_layernorm(a, stream));
}

size_t cssd_layernorm_backward_workspace_bytes(int64_t rows, int64_t width) {
    if (check_norm(rows, width, CSSD_F32, CSSD_F32) != CSSD_OK) return 0;
    return cssd::layernorm_backward_workspace_bytes(rows, width);
}

int cssd_layernorm_backward(int64_t rows, int64_t width, int xtype, int wtype, const void* dy, const void* x,
                            const void* weight, const float* mean, const float* rstd, void* gx, void* gweight,
                            void* gbias, void* workspace, size_t workspace_bytes, cssd_stream_t stream_) {
    int s = check_norm(rows, width, xtype, wtype);
    if (s != CSSD_OK) return s;
    if (!dy || !x || !mean || !rstd || !gx) return CSSD_ERR_NULL;
    if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(weight, 16) || !aligned(gx, 16) || !aligned(gweight, 16) ||
        !aligned(gbias, 16) || !aligned(workspace, 16) || !aligned(mean, 4) || !aligned(rstd, 4))
        return CSSD_ERR_ALIGN;
    const size_t need = cssd::layernorm_backward_workspace_bytes(rows, width);
    if (workspace && workspace_bytes < need) return CSSD_ERR_WORKSPACE;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    int dev = 0;
    if ((s = stream_device(stream, &dev)) != CSSD_OK) return s;
    if ((s = check_all_device(dev, dy, x, weight, (const void*)mean, (const void*)rstd, (const void*)gx,
                              (const void*)gweight, (const void*)gbias, (const void*)workspace)) != CSSD_OK)
        return s;
    Workspace ws(workspace, need, stream);
    if (ws.status != CSSD_OK) return ws.status;
    cssd::NormArgs a{};
    a.rows = rows;
    a.width = width;
    a.xtype = xtype;
    a.wtype = wtype;
    a.x = x;
    a.weight = weight;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.dy = dy;
    a.gx = gx;
    a.gweight = gweight;
    a.gbias = gbias;
    return status_of(cssd::launch_layernorm_backward(a, ws.p, stream));
}

static int check_linattn_dims(const cssd_delta_dims* d, int dtype, bool need_seq) {
    const int s = check_delta_dims(d, dtype, need_seq);
    if (s != CSSD_OK || !need_seq) return s;
    // tokens, rounded up to chunks of 128, in 32 bits
    if (d->seqlen > kMaxInt - 127) return CSSD_ERR_DIMS;
    // (row and head, chunk) in 32 bits, for the smallest chunk
    return product_fits(d->batch * d->nheads, (d->seqlen + 31) / 32, kMaxInt) ? CSSD_OK : CSSD_ERR_DIMS;
}

static cssd::LinattnArgs linattn_args(const cssd_delta_dims* d, int dtype) {
    cssd::LinattnArgs a{};
    a.Bz = d->batch;
    a.T = d->seqlen;
    a.H = d->nheads;
    a.KH = d->kheads;
    a.N = d->dstate;
    a.P = d->headdim;
    a.dtype = dtype;
    return a;
}

size_t cssd_linattn_workspace_bytes(const cssd_delta_dims* d, int dtype) {
    if (check_linattn_dims(d, dtype, true) != CSSD_OK) return 0;
    return cssd::linattn_workspace_bytes(linattn_args(d, dtype));
}

size_t cssd_linattn_backward_workspace_bytes(const cssd_delta_dims* d, int dtype) {
    if (check_linattn_dims(d, dtype, true) != CSSD_OK) return 0;
    return cssd::linattn_backward_workspace_bytes(linattn_args(d, dtype));
}

int cssd_linattn_forward(const cssd_delta_dims* d, int dtype, const void* q, const void* k, const void* v, const float* g,
                         int g_tokens, float scale, const float* h0, const int32_t* lens, void* o, float* h_final,
                         void* workspace, size_t workspace_bytes, cssd_stream_t stream_) {
    int s = check_linattn_dims(d, dtype, true);
    if (s != CSSD_OK) return s;
    if (!q || !k || !v || !g || !o) return CSSD_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(h0, 16) ||
        !aligned(h_final, 16) || !aligned(workspace, 16) || !aligned(g, 4) || !aligned(lens, 4))
        return CSSD_ERR_ALIGN;
    cssd::LinattnArgs a = linattn_args(d, dtype);
    const size_t need = cssd::linattn_workspace_bytes(a);
    if (workspace && workspace_bytes < need) return CSSD_ERR_WORKSPACE;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    int dev = 0;
    if ((s = stream_device(stream, &dev)) != CSSD_OK) return s;
    if ((s = check_all_device(dev, q, k, v, (const void*)g, (const void*)h0, (const void*)lens, (const void*)o,
                              (const void*)h_final, (const void*)workspace)) != CSSD_OK)
        return s;
    Workspace ws(workspace, need, stream);
    if (ws.status != CSSD_OK) return ws.status;
    a.scale = scale;
    a.q = q;
    a.k = k;
    a.v = v;
    a.g = g;
    a.g_tokens = g_tokens != 0;
    a.h0 = h0;
    a.lens = lens;
    a.o = o;
    a.h_final = h_final;
    return status_of(cssd::launch_linattn_forward(a, ws.p, stream));
}

int cssd_linattn_backward(const cssd_delta_dims* d, int dtype, const void* q, const void* k, const void* v, const float* g,
                          int g_tokens, float scale, const float* h0, const int32_t* lens, const void* dout,
                          const float* dh_final, void* gq, void* gk, void* gv, float* gg, float* gh0, void* workspace,
                          size_t workspace_bytes, cssd_stream_t stream_) {
    int s = check_linattn_dims(d, dtype, true);
    if (s != CSSD_OK) return s;
    if (!q || !k || !v || !g || !dout || !gq || !gk || !gv) return CSSD_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(dout, 16) || !aligned(h0, 16) ||
        !aligned(dh_final, 16) || !aligned(gq, 16) || !aligned(gk, 16) || !aligned(gv, 16) || !aligned(gh0, 16) ||
        !aligned(workspace, 16) || !aligned(g, 4) || !aligned(lens, 4) || !aligned(gg, 4))
        return CSSD_ERR_ALIGN;
    cssd::LinattnArgs a = linattn_args(d, dtype);
    const size_t need = cssd::linattn_backward_workspace_bytes(a);
    if (workspace && workspace_bytes < need) return CSSD_ERR_WORKSPACE;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    int dev = 0;
    if ((s = stream_device(stream, &dev)) != CSSD_OK) return s;
    if ((s = check_all_device(dev, q, k, v, (const void*)g, (const void*)h0, (const void*)lens, dout, (const void*)dh_final,
                              (const void*)gq, (const void*)gk, (const void*)gv, (const void*)gg, (const void*)gh0,
                              (const void*)workspace)) != CSSD_OK)
        return s;
    Workspace ws(workspace, need, stream);
    if (ws.status != CSSD_OK) return ws.status;
    a.scale = scale;
    a.q = q;
    a.k = k;
    a.v = v;
    a.g = g;
    a.g_tokens = g_tokens != 0;
    a.h0 = h0;
    a.lens = lens;
    a.dout = dout;
    a.dh_final = dh_final;
    a.gq = gq;
    a.gk = gk;
    a.gv = gv;
    a.gg = gg;
    a.gh0 = gh0;
    return status_of(cssd::launch_linattn_backward(a, ws.p, stream));
}

int cssd_linattn_step(const cssd_delta_dims* d, int dtype, float* h, int64_t nslots, const int32_t* slots, const void* q,
                      const void* k, const void* v, const float* g, int g_tokens, float scale, void* o,
                      cssd_stream_t stream_) {
    int s = check_linattn_dims(d, dtype, false);
    if (s != CSSD_OK) return s;
    if (nslots <= 0 || (!slots && nslots < d->batch)) return CSSD_ERR_DIMS;
    if (!h || !q || !k || !v || !g || !o) return CSSD_ERR_NULL;
    if (!aligned(h, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(g, 4) ||
        !aligned(slots, 4))
        return CSSD_ERR_ALIGN;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    int dev = 0;
    if ((s = stream_device(stream, &dev)) != CSSD_OK) return s;
    if ((s = check_all_device(dev, (const void*)h, (const void*)slots, q, k, v, (const void*)g, (const void*)o)) != CSSD_OK)
        return s;
    cssd::LinattnStepArgs a{};
    a.Bz = d->batch;
    a.H = d->nheads;
    a.KH = d->kheads;
    a.N = d->dstate;
    a.P = d->headdim;
    a.nslots = nslots;
    a.dtype = dtype;
    a.scale = scale;
    a.h = h;
    a.slots = slots;
    a.q = q;
    a.k = k;
    a.v = v;
    a.g = g;
    a.g_tokens = g_tokens != 0;
    a.o = o;
    return status_of(cssd::launch_linattn_step(a, stream));
}

static int check_kind(int kind) { return kind == CSSD_RMS || kind == CSSD_LAYER ? CSSD_OK : CSSD_ERR_UNSUPPORTED; }

static int check_add_norm(int64_t rows, int64_t width, int xtype, int rtype, int wtype, int kind) {
    const int s = check_norm(rows, width, xtype, wtype);
    if (s != CSSD_OK) return s;
    if (rtype != xtype && rtype != CSSD_F32) return CSSD_ERR_UNSUPPORTED;
    return check_kind(kind);
}

int cssd_add_norm(int64_t rows, int64_t width, int xtype, int rtype, int wtype, int kind, const void* x,
                  const void* residual, const void* scale, float alpha, const void* weight, const void* bias, float eps,
                  void* s_out, void* y, float* mean, float* rstd, cssd_stream_t stream_) {
    int s = check_add_norm(rows, width, xtype, rtype, wtype, kind);
    if (s != CSSD_OK) return s;
    if (!(eps >= 0.f)) return CSSD_ERR_DIMS;
    if (!x || !residual || !s_out || !y) return CSSD_ERR_NULL;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(scale, 16) || !aligned(weight, 16) || !aligned(bias, 16) ||
        !aligned(s_out, 16) || !aligned(y, 16) || !aligned(mean, 4) || !aligned(rstd, 4))
        return CSSD_ERR_ALIGN;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    int dev = 0;
    if ((s = stream_device(stream, &dev)) != CSSD_OK) return s;
    if ((s = check_all_device(dev, x, residual, scale, weight, bias, (const void*)s_out, (const void*)y, (const void*)mean,
                              (const void*)rstd)) != CSSD_OK)
        return s;
    cssd::AddNormArgs a{};
    a.rows = rows;
    a.width = width;
    a.xtype = xtype;
    a.rtype = rtype;
    a.wtype = wtype;
    a.layer = kind == CSSD_LAYER;
    a.alpha = alpha;
    a.eps = eps;
    a.x = x;
    a.residual = residual;
    a.scale = scale;
    a.weight = weight;
    a.bias = bias;
    a.s = s_out;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    return status_of(cssd::launch_add_norm(a, stream));
}

size_t cssd_add_norm_backward_workspace_bytes(int64_t rows, int64_t width) {
    if (check_norm(rows, width, CSSD_F32, CSSD_F32) != CSSD_OK) return 0;
    return cssd::add_norm_backward_workspace_bytes(rows, width);
}

int cssd_add_norm_backward(int64_t rows, int64_t width, int xtype, int rtype, int wtype, int kind, const void* dy,
                           const void* ds, const void* x, const void* s_in, const void* scale, float alpha,
                           const void* weight, const float* mean, const float* rstd, void* gx, void* gresidual,
                           void* gscale, void* gweight, void* gbias, void* workspace, size_t workspace_bytes,
                           cssd_stream_t stream_) {
    int s = check_add_norm(rows, width, xtype, rtype, wtype, kind);
    if (s != CSSD_OK) return s;
    if (!dy || !s_in || !rstd || !gx || !gresidual || (kind == CSSD_LAYER && !mean) || (gscale && !x)) return CSSD_ERR_NULL;
    if (!aligned(dy, 16) || !aligned(ds, 16) || !aligned(x, 16) || !aligned(s_in, 16) || !aligned(scale, 16) ||
        !aligned(weight, 16) || !aligned(gx, 16) || !aligned(gresidual, 16) || !aligned(gscale, 16) ||
        !aligned(gweight, 16) || !aligned(gbias, 16) || !aligned(workspace, 16) || !aligned(mean, 4) || !aligned(rstd, 4))
        return CSSD_ERR_ALIGN;
    const size_t need = cssd::add_norm_backward_workspace_bytes(rows, width);
    if (workspace && workspace_bytes < need) return CSSD_ERR_WORKSPACE;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    int dev = 0;
    if ((s = stream_device(stream, &dev)) != CSSD_OK) return s;
    if ((s = check_all_device(dev, dy, ds, x, s_in, scale, weight, (const void*)mean, (const void*)rstd, (const void*)gx,
                              (const void*)gresidual, (const void*)gscale, (const void*)gweight, (const void*)gbias,
                              (const void*)workspace)) != CSSD_OK)
        return s;
    Workspace ws(workspace, need, stream);
    if (ws.status != CSSD_OK) return ws.status;
    cssd::AddNormArgs a{};
    a.rows = rows;
    a.width = width;
    a.xtype = xtype;
    a.rtype = rtype;
    a.wtype = wtype;
    a.layer = kind == CSSD_LAYER;
    a.alpha = alpha;
    a.x = x;
    a.scale = scale;
    a.weight = weight;
    a.s = const_cast<void*>(s_in);
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.dy = dy;
    a.ds = ds;
    a.gx = gx;
    a.gresidual = gresidual;
    a.gscale = gscale;
    a.gweight = gweight;
    a.gbias = gbias;
    return status_of(cssd::launch_add_norm_backward(a, ws.p, stream));
}

static int check_gated_norm(int64_t rows, int64_t width, int64_t group, int xtype, int wtype, int kind) {
    const int s = check_norm(rows, width, xtype, wtype);
    if (s != CSSD_OK) return s;
    if (group <= 0 || width % group) return CSSD_ERR_DIMS;
    // (row and group in 32 bits)
    if (!product_fits(rows, width / group, kMaxInt)) return CSSD_ERR_DIMS;
    return check_kind(kind);
}

int cssd_gated_norm(int64_t rows, int64_t width, int64_t group, int xtype, int wtype, int kind, int gate_first,
                    const void* x, const void* z, const void* weight, const void* bias, float eps, void* y, float* mean,
                    float* rstd, cssd_stream_t stream_) {
    int s = check_gated_norm(rows, width, group, xtype, wtype, kind);
    if (s != CSSD_OK) return s;
    if (!(eps >= 0.f)) return CSSD_ERR_DIMS;
    if (!x || !z || !y) return CSSD_ERR_NULL;
    if (!aligned(x, 16) || !aligned(z, 16) || !aligned(weight, 16) || !aligned(bias, 16) || !aligned(y, 16) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return CSSD_ERR_ALIGN;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    int dev = 0;
    if ((s = stream_device(stream, &dev)) != CSSD_OK) return s;
    if ((s = check_all_device(dev, x, z, weight, bias, (const void*)y, (const void*)mean, (const void*)rstd)) != CSSD_OK)
        return s;
    cssd::GatedNormArgs a{};
    a.rows = rows;
    a.width = width;
    a.group = group;
    a.xtype = xtype;
    a.wtype = wtype;
    a.layer = kind == CSSD_LAYER;
    a.gate_first = gate_first != 0;
    a.eps = eps;
    a.x = x;
    a.z = z;
    a.weight = weight;
    a.bias = bias;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    return status_of(cssd::launch_gated_norm(a, stream));
}

size_t cssd_gated_norm_backward_workspace_bytes(int64_t rows, int64_t width, int64_t group) {
    if (check_gated_norm(rows, width, group, CSSD_F32, CSSD_F32, CSSD_RMS) != CSSD_OK) return 0;
    return cssd::gated_norm_backward_workspace_bytes(rows, width, group);
}

int cssd_gated_norm_backward(int64_t rows, int64_t width, int64_t group, int xtype, int wtype, int kind, int gate_first,
                             const void* dy, const void* x, const void* z, const void* weight, const void* bias,
                             const float* mean, const float* rstd, void* gx, void* gz, void* gweight, void* gbias,
                             void* workspace, size_t workspace_bytes, cssd_stream_t stream_) {
    int s = check_gated_norm(rows, width, group, xtype, wtype, kind);
    if (s != CSSD_OK) return s;
    if (!dy || !x || !z || !rstd || !gx || !gz || (kind == CSSD_LAYER && !mean)) return CSSD_ERR_NULL;
    if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(z, 16) || !aligned(weight, 16) || !aligned(bias, 16) ||
        !aligned(gx, 16) || !aligned(gz, 16) || !aligned(gweight, 16) || !aligned(gbias, 16) || !aligned(workspace, 16) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return CSSD_ERR_ALIGN;
    const size_t need = cssd::gated_norm_backward_workspace_bytes(rows, width, group);
    if (workspace && workspace_bytes < need) return CSSD_ERR_WORKSPACE;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    int dev = 0;
    if ((s = stream_device(stream, &dev)) != CSSD_OK) return s;
    if ((s = check_all_device(dev, dy, x, z, weight, bias, (const void*)mean, (const void*)rstd, (const void*)gx,
                              (const void*)gz, (const void*)gweight, (const void*)gbias, (const void*)workspace)) != CSSD_OK)
        return s;
    Workspace ws(workspace, need, stream);
    if (ws.status != CSSD_OK) return ws.status;
    cssd::GatedNormArgs a{};
    a.rows = rows;
    a.width = width;
    a.group = group;
    a.xtype = xtype;
    a.wtype = wtype;
    a.layer = kind == CSSD_LAYER;
    a.gate_first = gate_first != 0;
    a.x = x;
    a.z = z;
    a.weight = weight;
    a.bias = bias;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.dy = dy;
    a.gx = gx;
    a.gz = gz;
    a.gweight = gweight;
    a.gbias = gbias;
    return status_of(cssd::launch_gated_norm_backward(a, ws.p, stream));
}

}  // extern "C"
