// mixer_api.cu -- the C ABI of the mixer-block operators (declared in
// include/ssd.h): argument checks on the host, before any launch.
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/ssd.h"
#include "mixer.cuh"

namespace {

ssd_status refuse(ssd_status s, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
ssd_status refuse(ssd_status s, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    ssd::set_last_error(buf);
    return s;
}
ssd_status done(cudaError_t e, const char *what) {
    return e == cudaSuccess ? SSD_OK : refuse(SSD_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool valid(ssd_dtype d) { return d == SSD_F32 || d == SSD_BF16; }
size_t size_of(ssd_dtype d) { return d == SSD_BF16 ? 2 : 4; }
bool on(const void *p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Rows that may be strided need their element's alignment; contiguous tensors 16 bytes.
#define NEED_ELEM(p, dt) \
    if (!on(p, size_of(dt))) return refuse(SSD_ERR_INVALID_ARG, #p " is not aligned to its elements")
#define NEED_16(p) \
    if (!on(p, 16)) return refuse(SSD_ERR_INVALID_ARG, #p " must be 16-byte aligned")
#define NEED(p) \
    if (!(p)) return refuse(SSD_ERR_INVALID_ARG, #p " must be non-null")
#define NEED_STRIDE(ld, width) \
    if ((ld) < (width)) return refuse(SSD_ERR_INVALID_ARG, #ld " (%lld) is below the row's width (%lld)", (long long)(ld), (long long)(width))

constexpr int kMaxRows = 1 << 30;
constexpr int kMaxBatch = 65535;

ssd_status check_packed(int tokens, int nseq, const int *cu) {
    if (tokens < 0 || nseq < 0) return refuse(SSD_ERR_INVALID_ARG, "tokens (%d) and nseq (%d) must be >= 0", tokens, nseq);
    if (tokens > kMaxRows || nseq > kMaxRows) return refuse(SSD_ERR_UNSUPPORTED, "more than 2^30 tokens or sequences");
    if (tokens > 0 && nseq > 0) {
        NEED(cu);
        if (!on(cu, 4)) return refuse(SSD_ERR_INVALID_ARG, "cu_seqlens is not aligned to its elements");
    }
    return SSD_OK;
}
ssd_status check_slots(const void *state, const int *slots, int nslots, int rows) {
    if (!state) return SSD_OK;
    NEED_16(state);
    if (!on(slots, 4)) return refuse(SSD_ERR_INVALID_ARG, "slots is not aligned to its elements");
    if (nslots < 0 || (!slots && nslots < rows))
        return refuse(SSD_ERR_INVALID_ARG, "%d states for %d sequences, and no slots that choose among them", nslots, rows);
    return SSD_OK;
}

ssd_status check_conv(ssd_dtype io, int x_channels, int bc_channels, int width, long long ld) {
    if (!valid(io)) return refuse(SSD_ERR_INVALID_ARG, "io_dtype must be SSD_F32 or SSD_BF16");
    if (x_channels <= 0 || bc_channels < 0) return refuse(SSD_ERR_INVALID_ARG, "x_channels must be > 0 and bc_channels >= 0");
    if (width < 1 || width > 8) return refuse(SSD_ERR_UNSUPPORTED, "width must be in 1..8 (got %d)", width);
    const long long ctot = (long long)x_channels + 2LL * bc_channels;
    if (ctot > 1 << 20) return refuse(SSD_ERR_UNSUPPORTED, "more than 2^20 channels");
    NEED_STRIDE(ld, ctot);
    return SSD_OK;
}

ssd_status check_sel(ssd_dtype io, int channels, int ngroups, int dstate) {
    if (!valid(io)) return refuse(SSD_ERR_INVALID_ARG, "io_dtype must be SSD_F32 or SSD_BF16");
    if (channels <= 0 || ngroups <= 0 || dstate <= 0)
        return refuse(SSD_ERR_INVALID_ARG, "channels (%d), ngroups (%d) and dstate (%d) must be > 0", channels, ngroups, dstate);
    if (channels % ngroups) return refuse(SSD_ERR_INVALID_ARG, "ngroups (%d) must divide channels (%d)", ngroups, channels);
    if (dstate > ssd::SEL_MAX_DSTATE)
        return refuse(SSD_ERR_UNSUPPORTED, "dstate must be at most %d (got %d)", ssd::SEL_MAX_DSTATE, dstate);
    // grid.y: a block takes at least 16 channels of one group (dstate 64, four lanes or more a channel)
    if (ngroups * ((channels / ngroups + 15LL) / 16) > 65535) return refuse(SSD_ERR_UNSUPPORTED, "too many channels for the grid");
    return SSD_OK;
}

// The inputs every selective scan call has (any_rows: some are read).
ssd_status sel_inputs(const ssd_sel_args *a, ssd::SelCall &c, bool any_rows = true) {
    NEED(a);
    ssd_status s = check_sel(a->io_dtype, a->channels, a->ngroups, a->dstate);
    if (s != SSD_OK) return s;
    const ssd_dtype io = a->io_dtype;
    const void *x = a->x, *dt = a->dt, *z = a->z, *B = a->B, *C = a->C;
    const float *A = a->A, *D = a->D, *dt_bias = a->dt_bias;
    NEED(A);
    if (any_rows) {
        NEED(x);
        NEED(dt);
        NEED(B);
        NEED(C);
    }
    NEED_ELEM(x, io);
    NEED_ELEM(dt, io);
    NEED_ELEM(z, io);
    NEED_ELEM(B, io);
    NEED_ELEM(C, io);
    NEED_16(A);
    NEED_16(D);
    NEED_16(dt_bias);
    const long long bc = (long long)a->ngroups * a->dstate;
    NEED_STRIDE(a->x_stride, a->channels);
    NEED_STRIDE(a->dt_stride, a->channels);
    if (z) NEED_STRIDE(a->z_stride, a->channels);
    NEED_STRIDE(a->b_stride, bc);
    NEED_STRIDE(a->c_stride, bc);
    c = ssd::SelCall{};
    c.x = x, c.dt = dt, c.z = z, c.B = B, c.C = C;
    c.ld_x = a->x_stride, c.ld_dt = a->dt_stride, c.ld_z = a->z_stride, c.ld_b = a->b_stride, c.ld_c = a->c_stride;
    c.A = A, c.D = D, c.dt_bias = dt_bias;
    c.bf16 = io == SSD_BF16;
    c.softplus = a->softplus, c.channels = a->channels, c.groups = a->ngroups, c.dstate = a->dstate;
    return SSD_OK;
}

ssd_status norm_sizes(ssd_dtype io, int rows, int width, int ngroups, float eps) {
    if (!valid(io)) return refuse(SSD_ERR_INVALID_ARG, "io_dtype must be SSD_F32 or SSD_BF16");
    if (rows < 0 || width <= 0 || ngroups <= 0) return refuse(SSD_ERR_INVALID_ARG, "rows must be >= 0, width and ngroups > 0");
    if (width % ngroups) return refuse(SSD_ERR_INVALID_ARG, "ngroups (%d) must divide width (%d)", ngroups, width);
    if (width / ngroups > ssd::NORM_MAX_WIDTH)
        return refuse(SSD_ERR_UNSUPPORTED, "a normalised group has at most %d channels (got %d)", ssd::NORM_MAX_WIDTH, width / ngroups);
    if (rows > kMaxRows || ngroups > 65535) return refuse(SSD_ERR_UNSUPPORTED, "more than 2^30 rows or 65535 groups");
    if (!(eps >= 0.f)) return refuse(SSD_ERR_INVALID_ARG, "eps must be >= 0");
    return SSD_OK;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------ convolution

ssd_status ssd_conv1d_varlen(const void *xbc, long long xbc_stride, const float *weight, const float *bias,
                             const int *cu_seqlens, void *conv_state, const int *slots, const unsigned char *has_init,
                             void *x_out, void *B_out, void *C_out, ssd_dtype io_dtype, int tokens, int nseq, int nslots,
                             int x_channels, int bc_channels, int width, int silu, void *stream) {
    ssd_status s = check_conv(io_dtype, x_channels, bc_channels, width, xbc_stride);
    if (s == SSD_OK) s = check_packed(tokens, nseq, cu_seqlens);
    if (s == SSD_OK) s = check_slots(conv_state, slots, nslots, nseq);
    if (s != SSD_OK || tokens == 0 || nseq == 0) return s;
    NEED(xbc);
    NEED(weight);
    NEED(x_out);
    if (bc_channels > 0) {
        NEED(B_out);
        NEED(C_out);
    }
    NEED_ELEM(xbc, io_dtype);
    NEED_16(weight);
    NEED_16(bias);
    NEED_16(x_out);
    NEED_16(B_out);
    NEED_16(C_out);
    int *err = ssd::device_error_word();
    if (!err) return SSD_ERR_CUDA;
    const ssd::ConvCall c{xbc, xbc_stride, weight, bias, x_out, B_out, C_out, conv_state, nullptr, nullptr, nullptr,
                          io_dtype == SSD_BF16, x_channels, bc_channels, width, silu != 0,
                          ssd::Packed{cu_seqlens, nseq, tokens, slots, nslots, has_init, err}};
    return done(ssd::launch_conv_varlen(c, static_cast<cudaStream_t>(stream)), "conv1d_varlen launch");
}

ssd_status ssd_conv1d_update(void *conv_state, const int *slots, const void *xbc, long long xbc_stride, const float *weight,
                             const float *bias, void *x_out, void *B_out, void *C_out, ssd_dtype io_dtype, int batch,
                             int nslots, int x_channels, int bc_channels, int width, int silu, void *stream) {
    ssd_status s = check_conv(io_dtype, x_channels, bc_channels, width, xbc_stride);
    if (s == SSD_OK && (batch < 0 || batch > kMaxBatch))
        s = refuse(batch < 0 ? SSD_ERR_INVALID_ARG : SSD_ERR_UNSUPPORTED, "batch must be in 0..%d", kMaxBatch);
    if (s == SSD_OK) s = check_slots(conv_state, slots, nslots, batch);
    if (s != SSD_OK || batch == 0) return s;
    if (width > 1) NEED(conv_state);
    if (!on(slots, 4)) return refuse(SSD_ERR_INVALID_ARG, "slots is not aligned to its elements");
    NEED(xbc);
    NEED(weight);
    NEED(x_out);
    if (bc_channels > 0) {
        NEED(B_out);
        NEED(C_out);
    }
    NEED_ELEM(xbc, io_dtype);
    NEED_16(weight);
    NEED_16(bias);
    NEED_16(x_out);
    NEED_16(B_out);
    NEED_16(C_out);
    int *err = ssd::device_error_word();
    if (!err) return SSD_ERR_CUDA;
    const ssd::ConvCall c{xbc, xbc_stride, weight, bias, x_out, B_out, C_out, conv_state, nullptr, nullptr, nullptr,
                          io_dtype == SSD_BF16, x_channels, bc_channels, width, silu != 0,
                          ssd::Packed{nullptr, batch, batch, slots, nslots, nullptr, err}};
    return done(ssd::launch_conv_update(c, batch, static_cast<cudaStream_t>(stream)), "conv1d_update launch");
}

size_t ssd_conv1d_bwd_workspace_size(int tokens, int channels, int width) {
    if (tokens < 0 || tokens > kMaxRows || channels <= 0 || channels > 1 << 20 || width < 1 || width > 8) return SSD_WORKSPACE_INVALID;
    return ssd::conv_bwd_workspace(tokens, channels, width);
}

ssd_status ssd_conv1d_bwd(const void *xbc, long long xbc_stride, const float *weight, const float *bias,
                          const int *cu_seqlens, const void *dx_out, const void *dB_out, const void *dC_out, void *dxbc,
                          float *dweight, float *dbias, ssd_dtype io_dtype, int tokens, int nseq, int x_channels,
                          int bc_channels, int width, int silu, void *workspace, size_t workspace_bytes, void *stream) {
    ssd_status s = check_conv(io_dtype, x_channels, bc_channels, width, xbc_stride);
    if (s == SSD_OK) s = check_packed(tokens, nseq, cu_seqlens);
    if (s != SSD_OK) return s;
    NEED(dweight);
    NEED_16(dweight);
    NEED_16(dbias);
    if (tokens > 0) {
        NEED(xbc);
        NEED(weight);
        NEED(dx_out);
        NEED(dxbc);
        if (bc_channels > 0) {
            NEED(dB_out);
            NEED(dC_out);
        }
    }
    NEED_ELEM(xbc, io_dtype);
    NEED_16(weight);
    NEED_16(bias);
    NEED_16(dx_out);
    NEED_16(dB_out);
    NEED_16(dC_out);
    NEED_16(dxbc);
    const size_t need = ssd::conv_bwd_workspace(tokens, x_channels + 2 * bc_channels, width);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return refuse(SSD_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need, workspace ? workspace_bytes : (size_t)0);
    NEED_16(workspace);
    int *err = ssd::device_error_word();
    if (!err) return SSD_ERR_CUDA;
    const ssd::ConvCall c{xbc, xbc_stride, weight, bias, const_cast<void *>(dx_out), const_cast<void *>(dB_out),
                          const_cast<void *>(dC_out), nullptr, dxbc, dweight, dbias, io_dtype == SSD_BF16, x_channels,
                          bc_channels, width, silu != 0, ssd::Packed{cu_seqlens, nseq, tokens, nullptr, 0, nullptr, err}};
    return done(ssd::launch_conv_bwd(c, static_cast<float *>(workspace), static_cast<cudaStream_t>(stream)), "conv1d_bwd launch");
}

// --------------------------------------------------------------- selective scan

size_t ssd_selective_scan_chunk_states(int tokens, int nseq) {
    if (tokens < 0 || nseq < 0 || tokens > kMaxRows || nseq > kMaxRows) return SSD_WORKSPACE_INVALID;
    return (size_t)(tokens / ssd::SEL_CHUNK) + nseq;
}

size_t ssd_selective_scan_workspace_size(int tokens, int nseq, int channels, int dstate) {
    if (tokens < 0 || nseq < 0 || tokens > kMaxRows || nseq > kMaxRows || check_sel(SSD_F32, channels, 1, dstate) != SSD_OK)
        return SSD_WORKSPACE_INVALID;
    return ssd::sel_fwd_workspace(tokens, nseq, channels, dstate);
}

ssd_status ssd_selective_scan_varlen(const ssd_sel_args *args, const int *cu_seqlens, float *state, const int *slots,
                                     const unsigned char *has_init, float *chunk_states, void *y, int tokens, int nseq,
                                     int nslots, void *workspace, size_t workspace_bytes, void *stream) {
    ssd_status s = check_packed(tokens, nseq, cu_seqlens);
    if (s == SSD_OK) s = check_slots(state, slots, nslots, nseq);
    if (s != SSD_OK || tokens == 0 || nseq == 0) return s;
    ssd::SelCall c;
    s = sel_inputs(args, c);
    if (s != SSD_OK) return s;
    NEED(y);
    NEED_16(y);
    NEED_16(chunk_states);
    const size_t need = ssd::sel_fwd_workspace(tokens, nseq, c.channels, c.dstate);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return refuse(SSD_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need, workspace ? workspace_bytes : (size_t)0);
    NEED_16(workspace);
    int *err = ssd::device_error_word();
    if (!err) return SSD_ERR_CUDA;
    c.state = state, c.chunk_states = chunk_states, c.y = y;
    c.seq = ssd::Packed{cu_seqlens, nseq, tokens, slots, nslots, has_init, err};
    return done(ssd::launch_sel_varlen(c, static_cast<float *>(workspace), static_cast<cudaStream_t>(stream)), "selective_scan_varlen launch");
}

ssd_status ssd_selective_state_update(const ssd_sel_args *args, float *state, const int *slots, void *y, int batch,
                                      int nslots, void *stream) {
    if (batch < 0 || batch > kMaxBatch)
        return refuse(batch < 0 ? SSD_ERR_INVALID_ARG : SSD_ERR_UNSUPPORTED, "batch must be in 0..%d", kMaxBatch);
    ssd_status s = check_slots(state, slots, nslots, batch);
    if (s != SSD_OK || batch == 0) return s;
    ssd::SelCall c;
    s = sel_inputs(args, c);
    if (s != SSD_OK) return s;
    NEED(state);
    NEED(y);
    NEED_16(y);
    int *err = ssd::device_error_word();
    if (!err) return SSD_ERR_CUDA;
    c.state = state, c.y = y;
    c.seq = ssd::Packed{nullptr, batch, batch, slots, nslots, nullptr, err};
    return done(ssd::launch_sel_update(c, batch, static_cast<cudaStream_t>(stream)), "selective_state_update launch");
}

size_t ssd_selective_scan_bwd_workspace_size(int tokens, int nseq, int channels, int ngroups, int dstate) {
    if (tokens < 0 || nseq < 0 || tokens > kMaxRows || nseq > kMaxRows) return SSD_WORKSPACE_INVALID;
    if (check_sel(SSD_F32, channels, ngroups, dstate) != SSD_OK) return SSD_WORKSPACE_INVALID;
    return ssd::sel_bwd_workspace(tokens, nseq, channels, ngroups, dstate);
}

ssd_status ssd_selective_scan_bwd(const ssd_sel_args *args, const int *cu_seqlens, const void *dy, const float *chunk_states,
                                  void *dx, void *ddt, void *dz, void *dB, void *dC, float *dA, float *dD, float *ddt_bias,
                                  int tokens, int nseq, void *workspace, size_t workspace_bytes, void *stream) {
    ssd_status s = check_packed(tokens, nseq, cu_seqlens);
    if (s != SSD_OK) return s;
    ssd::SelCall c;
    s = sel_inputs(args, c, tokens > 0);
    if (s != SSD_OK) return s;
    NEED(dA);
    if (tokens > 0) {
        NEED(dy);
        NEED(dx);
        NEED(ddt);
        NEED(dB);
        NEED(dC);
        if (c.z) NEED(dz);
        if (nseq > 0) NEED(chunk_states);
    }
    for (const void *p : {dy, (const void *)chunk_states, (const void *)dx, (const void *)ddt, (const void *)dz,
                          (const void *)dB, (const void *)dC, (const void *)dA, (const void *)dD, (const void *)ddt_bias,
                          (const void *)workspace})
        NEED_16(p);
    const size_t need = ssd::sel_bwd_workspace(tokens, nseq, c.channels, c.groups, c.dstate);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return refuse(SSD_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need, workspace ? workspace_bytes : (size_t)0);
    int *err = ssd::device_error_word();
    if (!err) return SSD_ERR_CUDA;
    c.dy = dy, c.chunk_states = const_cast<float *>(chunk_states), c.dx = dx, c.ddt = ddt, c.dz = dz, c.dB = dB, c.dC = dC;
    c.dA = dA, c.dD = dD, c.dbias = ddt_bias;
    c.seq = ssd::Packed{cu_seqlens, nseq, tokens, nullptr, 0, nullptr, err};
    return done(ssd::launch_sel_bwd(c, workspace, static_cast<cudaStream_t>(stream)), "selective_scan_bwd launch");
}

// ------------------------------------------------------------------------ norms

ssd_status ssd_residual_rmsnorm(const void *x, long long x_stride, const void *residual, long long residual_stride,
                                const float *scale, const float *weight, void *out, void *residual_out,
                                ssd_dtype io_dtype, ssd_dtype residual_dtype, int rows, int width, float eps, void *stream) {
    ssd_status s = norm_sizes(io_dtype, rows, width, 1, eps);
    if (s != SSD_OK) return s;
    if (residual_dtype != SSD_F32 && residual_dtype != io_dtype)
        return refuse(SSD_ERR_INVALID_ARG, "residual_dtype must be SSD_F32 or io_dtype");
    if (rows == 0) return SSD_OK;
    NEED(x);
    NEED(weight);
    NEED(out);
    NEED_ELEM(x, io_dtype);
    NEED_ELEM(residual, residual_dtype);
    NEED_STRIDE(x_stride, width);
    if (residual) NEED_STRIDE(residual_stride, width);
    NEED_16(scale);
    NEED_16(weight);
    NEED_16(out);
    NEED_16(residual_out);
    ssd::NormCall c{};
    c.x = x, c.ld_x = x_stride, c.res = residual, c.ld_res = residual_stride, c.scale = scale, c.w = weight, c.out = out,
    c.res_out = residual_out, c.bf16 = io_dtype == SSD_BF16, c.res_bf16 = residual_dtype == SSD_BF16, c.rows = rows,
    c.width = width, c.groups = 1, c.eps = eps;
    return done(ssd::launch_norm_before(c, static_cast<cudaStream_t>(stream)), "residual_rmsnorm launch");
}

ssd_status ssd_gated_rmsnorm(const void *y, long long y_stride, const void *z, long long z_stride, const void *residual,
                             long long residual_stride, const float *scale, const float *weight, void *out,
                             ssd_dtype io_dtype, int rows, int width, int ngroups, int norm_before_gate, float eps,
                             void *stream) {
    ssd_status s = norm_sizes(io_dtype, rows, width, ngroups, eps);
    if (s != SSD_OK || rows == 0) return s;
    NEED(y);
    NEED(weight);
    NEED(out);
    NEED_ELEM(y, io_dtype);
    NEED_ELEM(z, io_dtype);
    NEED_ELEM(residual, io_dtype);
    NEED_STRIDE(y_stride, width);
    if (z) NEED_STRIDE(z_stride, width);
    if (residual) NEED_STRIDE(residual_stride, width);
    NEED_16(scale);
    NEED_16(weight);
    NEED_16(out);
    ssd::NormCall c{};
    c.x = y, c.ld_x = y_stride, c.z = z, c.ld_z = z_stride, c.res = residual, c.ld_res = residual_stride, c.scale = scale,
    c.w = weight, c.out = out, c.bf16 = io_dtype == SSD_BF16, c.res_bf16 = c.bf16, c.rows = rows, c.width = width,
    c.groups = ngroups, c.norm_first = norm_before_gate != 0, c.eps = eps;
    return done(ssd::launch_norm_after(c, static_cast<cudaStream_t>(stream)), "gated_rmsnorm launch");
}

size_t ssd_rmsnorm_bwd_workspace_size(int rows, int width) {
    if (rows < 0 || rows > kMaxRows || width <= 0) return SSD_WORKSPACE_INVALID;
    return ssd::norm_bwd_workspace(rows, width);
}

ssd_status ssd_residual_rmsnorm_bwd(const void *residual, long long residual_stride, const float *weight,
                                    const void *dout, const void *dresidual, const void *x, long long x_stride,
                                    const float *scale, void *dx, void *dresidual_in, float *dweight, float *dscale,
                                    ssd_dtype io_dtype, ssd_dtype residual_dtype, int rows, int width, float eps,
                                    void *workspace, size_t workspace_bytes, void *stream) {
    ssd_status s = norm_sizes(io_dtype, rows, width, 1, eps);
    if (s != SSD_OK) return s;
    if (residual_dtype != SSD_F32 && residual_dtype != io_dtype)
        return refuse(SSD_ERR_INVALID_ARG, "residual_dtype must be SSD_F32 or io_dtype");
    NEED(dweight);
    if (scale) NEED(dscale);
    if (rows > 0) {
        NEED(residual);
        NEED(weight);
        NEED(dout);
        if (scale) NEED(x);
        if (!dx && !dresidual_in) return refuse(SSD_ERR_INVALID_ARG, "dx or dresidual_in must be non-null");
        if (dx && dx == dresidual_in && (scale || residual_dtype != io_dtype))
            return refuse(SSD_ERR_INVALID_ARG, "dx and dresidual_in are one array, and scale or residual_dtype sets them apart");
        NEED_STRIDE(residual_stride, width);
        if (scale) NEED_STRIDE(x_stride, width);
    }
    NEED_ELEM(residual, residual_dtype);
    NEED_ELEM(x, io_dtype);
    for (const void *p : {(const void *)weight, dout, dresidual, (const void *)scale, (const void *)dx,
                          (const void *)dresidual_in, (const void *)dweight, (const void *)dscale, (const void *)workspace})
        NEED_16(p);
    const size_t need = ssd::norm_bwd_workspace(rows, width);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return refuse(SSD_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need, workspace ? workspace_bytes : (size_t)0);
    ssd::NormCall c{};
    c.x = scale ? x : nullptr, c.ld_x = x_stride, c.res = residual, c.ld_res = residual_stride, c.scale = scale, c.w = weight,
    c.dout = dout, c.dres = dresidual, c.dx = dx, c.dres_out = dresidual_in, c.dw = dweight, c.dscale = dscale,
    c.bf16 = io_dtype == SSD_BF16, c.res_bf16 = residual_dtype == SSD_BF16, c.rows = rows, c.width = width, c.groups = 1,
    c.eps = eps;
    return done(ssd::launch_norm_before_bwd(c, static_cast<float *>(workspace), static_cast<cudaStream_t>(stream)),
                "residual_rmsnorm_bwd launch");
}

ssd_status ssd_gated_rmsnorm_bwd(const void *y, long long y_stride, const void *z, long long z_stride, const float *weight,
                                 const void *dout, const float *scale, void *dy, void *dz, float *dweight, float *dscale,
                                 ssd_dtype io_dtype, int rows, int width, int ngroups, int norm_before_gate, float eps,
                                 void *workspace, size_t workspace_bytes, void *stream) {
    ssd_status s = norm_sizes(io_dtype, rows, width, ngroups, eps);
    if (s != SSD_OK) return s;
    NEED(dweight);
    if (scale) NEED(dscale);
    if (rows > 0) {
        NEED(y);
        NEED(weight);
        NEED(dout);
        NEED(dy);
        if (z) NEED(dz);
        NEED_STRIDE(y_stride, width);
        if (z) NEED_STRIDE(z_stride, width);
    }
    NEED_ELEM(y, io_dtype);
    NEED_ELEM(z, io_dtype);
    for (const void *p : {(const void *)weight, dout, (const void *)scale, (const void *)dy, (const void *)dz,
                          (const void *)dweight, (const void *)dscale, (const void *)workspace})
        NEED_16(p);
    const size_t need = ssd::norm_bwd_workspace(rows, width);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return refuse(SSD_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need, workspace ? workspace_bytes : (size_t)0);
    ssd::NormCall c{};
    c.x = y, c.ld_x = y_stride, c.z = z, c.ld_z = z_stride, c.scale = scale, c.w = weight, c.dout = dout, c.dx = dy, c.dz = dz,
    c.dw = dweight, c.dscale = dscale, c.bf16 = io_dtype == SSD_BF16, c.res_bf16 = c.bf16, c.rows = rows, c.width = width,
    c.groups = ngroups, c.norm_first = norm_before_gate != 0, c.eps = eps;
    return done(ssd::launch_norm_after_bwd(c, static_cast<float *>(workspace), static_cast<cudaStream_t>(stream)),
                "gated_rmsnorm_bwd launch");
}

}  // extern "C"
