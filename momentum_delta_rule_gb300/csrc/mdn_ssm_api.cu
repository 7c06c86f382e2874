// C ABI of the state-space layer's operators: argument validation and
// dispatch.  Declarations and the contract: include/mdn.h.
#include "mdn_ssm.cuh"

namespace mdn {
namespace {

constexpr long kMaxTokens = 0x3fffffffL;

int element_bytes(mdn_dtype dtype) { return dtype == MDN_BF16 ? 2 : 4; }
bool valid_dtype(mdn_dtype dtype) { return dtype == MDN_F32 || dtype == MDN_BF16; }

// Collects a call's pointers and checks them: required ones present, each
// aligned to its element, outputs distinct from everything else.
class Args {
  public:
    Args &in(const void *ptr, int align, bool required = true) {
        add(ptr, align, required);
        return *this;
    }
    Args &out(const void *ptr, int align, bool required = true, const void *may_be = nullptr) {
        if (ptr) {
            for (int i = 0; i < n_; ++i)
                if (seen_[i] == ptr && ptr != may_be) ok_ = false;
            for (int i = 0; i < n_out_; ++i)
                if (outs_[i] == ptr) ok_ = false;
            outs_[n_out_++] = ptr;
        }
        add(ptr, align, required);
        return *this;
    }
    bool ok() const { return ok_; }

  private:
    void add(const void *ptr, int align, bool required) {
        if (!ptr) {
            if (required) ok_ = false;
            return;
        }
        if ((uintptr_t)ptr % align) ok_ = false;
        seen_[n_++] = ptr;
    }
    const void *seen_[32];
    const void *outs_[16];
    int n_ = 0, n_out_ = 0;
    bool ok_ = true;
};

// Alignment of fp32 states [.., N]: whole packets of four where N has them.
int state_align(int N) { return N % 4 == 0 ? 16 : 4; }

bool batch_ok(const int32_t *cu, int n_seq, int B, int T) {
    if (B < 0 || T < 0 || n_seq < 0 || (long)B * T > kMaxTokens) return false;
    if (cu ? B != 1 : n_seq != B) return false;
    return !((uintptr_t)cu & 3u);
}

mdn_status finish(cudaError_t err) {
    if (err == cudaSuccess) return MDN_OK;
    cudaGetLastError();
    return MDN_ERR_CUDA;
}

bool bc_wide(const void *Bm, const void *Cm, int64_t ld_B, int64_t ld_C, int N, int el) {
    return N % 4 == 0 && rows_aligned(Bm, ld_B, el, 4 * el) && rows_aligned(Cm, ld_C, el, 4 * el);
}

bool workspace_ok(const void *ws, size_t bytes, size_t need) {
    return need == 0 || (ws && bytes >= need && !((uintptr_t)ws & 255u));
}

}  // namespace
}  // namespace mdn

using namespace mdn;

extern "C" {

mdn_status mdn_short_conv_fwd(const void *x, const float *w, const float *bias,
                              const void *state0, void *y, void *state_T,
                              const int32_t *cu_seqlens, int n_seq, int B, int T, int D,
                              int width, mdn_conv_act act, int64_t ld_x, mdn_dtype dtype,
                              void *stream) {
    if (D <= 0 || !valid_dtype(dtype) || !batch_ok(cu_seqlens, n_seq, B, T) || ld_x < D ||
        (act != MDN_CONV_NONE && act != MDN_CONV_SILU))
        return MDN_ERR_INVALID_ARG;
    if (width < 2 || width > 4) return MDN_ERR_UNSUPPORTED;
    const long L = (long)B * T;
    const int el = element_bytes(dtype);
    const bool some = L > 0;
    if (some && n_seq == 0) return MDN_ERR_INVALID_ARG;
    if (!Args().in(x, el, some).in(w, 4, some).in(bias, 4, false).in(state0, el, false)
             .out(y, el, some).out(state_T, el, false).ok())
        return MDN_ERR_INVALID_ARG;
    int *status = nullptr;
    const mdn_status st = current_device_status(&status);
    if (st != MDN_OK) return st;
    ConvProblem p = {};
    p.x = x; p.w = w; p.bias = bias; p.state0 = state0; p.y = y; p.state_T = state_T;
    p.cu = some ? cu_seqlens : nullptr; p.n_seq = n_seq; p.T = T; p.T_total = (int)L;
    p.D = D; p.width = width; p.act = act; p.ld_x = ld_x; p.dtype = dtype; p.status = status;
    return finish(launch_conv_fwd(p, static_cast<cudaStream_t>(stream)));
}

size_t mdn_short_conv_bwd_workspace_size(int T_total, int D, int width, mdn_dtype dtype) {
    if (T_total < 0 || D <= 0 || width < 2 || width > 4 || !valid_dtype(dtype)) return 0;
    return conv_bwd_workspace(T_total, D, width, dtype);
}

mdn_status mdn_short_conv_bwd(const void *x, const float *w, const float *bias,
                              const void *state0, const void *dy, const void *dstate_T, void *dx,
                              float *dw, float *dbias, void *dstate0, const int32_t *cu_seqlens,
                              int n_seq, int B, int T, int D, int width, mdn_conv_act act,
                              int64_t ld_x, int64_t ld_dy, mdn_dtype dtype, void *workspace,
                              size_t workspace_bytes, void *stream) {
    if (D <= 0 || !valid_dtype(dtype) || !batch_ok(cu_seqlens, n_seq, B, T) || ld_x < D ||
        ld_dy < D || (act != MDN_CONV_NONE && act != MDN_CONV_SILU))
        return MDN_ERR_INVALID_ARG;
    if (width < 2 || width > 4) return MDN_ERR_UNSUPPORTED;
    const long L = (long)B * T;
    const int el = element_bytes(dtype);
    const bool some = L > 0;
    if (some && n_seq == 0) return MDN_ERR_INVALID_ARG;
    if (!Args().in(x, el, some).in(w, 4, some).in(bias, 4, false).in(state0, el, false)
             .in(dy, el, some).in(dstate_T, el, false).out(dx, el, some).out(dw, 4)
             .out(dbias, 4, false).out(dstate0, el, false).ok())
        return MDN_ERR_INVALID_ARG;
    if (some && !workspace_ok(workspace, workspace_bytes,
                              mdn_short_conv_bwd_workspace_size((int)L, D, width, dtype)))
        return MDN_ERR_INVALID_ARG;
    int *status = nullptr;
    const mdn_status st = current_device_status(&status);
    if (st != MDN_OK) return st;
    ConvProblem p = {};
    p.x = x; p.dy = dy; p.w = w; p.bias = bias; p.state0 = state0; p.dstate_T = dstate_T;
    p.dx = dx; p.dstate0 = dstate0; p.dw = dw; p.dbias = dbias;
    p.partial = static_cast<float *>(workspace);
    p.cu = some ? cu_seqlens : nullptr; p.n_seq = n_seq; p.T = T; p.T_total = (int)L;
    p.D = D; p.width = width; p.act = act; p.ld_x = ld_x; p.ld_dy = ld_dy; p.dtype = dtype;
    p.status = status;
    return finish(launch_conv_bwd(p, static_cast<cudaStream_t>(stream)));
}

mdn_status mdn_short_conv_step(const void *x, const float *w, const float *bias,
                               const void *state, void *state_out, void *y, int N, int D,
                               int width, mdn_conv_act act, int64_t ld_x, mdn_dtype dtype,
                               void *stream) {
    if (N < 0 || D <= 0 || !valid_dtype(dtype) || ld_x < D ||
        (act != MDN_CONV_NONE && act != MDN_CONV_SILU))
        return MDN_ERR_INVALID_ARG;
    if (width < 2 || width > 4) return MDN_ERR_UNSUPPORTED;
    const int el = element_bytes(dtype);
    const bool some = N > 0;
    if (!Args().in(x, el, some).in(w, 4, some).in(bias, 4, false).in(state, el, some)
             .out(state_out, el, some, state).out(y, el, some).ok())
        return MDN_ERR_INVALID_ARG;
    int *status = nullptr;
    const mdn_status st = current_device_status(&status);
    if (st != MDN_OK) return st;
    ConvProblem p = {};
    p.x = x; p.w = w; p.bias = bias; p.state0 = state; p.state_T = state_out; p.y = y;
    p.n_seq = N; p.T = 1; p.T_total = N; p.D = D; p.width = width; p.act = act; p.ld_x = ld_x;
    p.dtype = dtype; p.status = status;
    return finish(launch_conv_step(p, static_cast<cudaStream_t>(stream)));
}

size_t mdn_ssm_state_slots(int n_seq, int B, int T, int packed) {
    if (n_seq < 0 || B < 0 || T < 0) return 0;
    if (packed) return (size_t)((long)B * T / MDN_SSM_CHUNK) + (size_t)n_seq;
    return (size_t)B * (size_t)(((long)T + MDN_SSM_CHUNK - 1) / MDN_SSM_CHUNK);
}

static bool scan_sizes_ok(int n_seq, int T_total, int D, int G, int N, mdn_dtype dtype) {
    return n_seq >= 0 && T_total >= 0 && D > 0 && G > 0 && D % G == 0 && N > 0 && N <= 128 &&
           valid_dtype(dtype);
}

size_t mdn_ssm_scan_fwd_workspace_size(int n_seq, int T_total, int D, int G, int N,
                                       mdn_dtype dtype) {
    if (!scan_sizes_ok(n_seq, T_total, D, G, N, dtype)) return 0;
    return scan_fwd_workspace(n_seq, T_total, D, G, N, dtype);
}
size_t mdn_ssm_scan_bwd_workspace_size(int n_seq, int T_total, int D, int G, int N,
                                       mdn_dtype dtype) {
    if (!scan_sizes_ok(n_seq, T_total, D, G, N, dtype)) return 0;
    return scan_bwd_workspace(n_seq, T_total, D, G, N, dtype);
}

mdn_status mdn_ssm_scan_fwd(const void *u, const void *dt, const float *A, const void *Bm,
                            const void *Cm, const float *D_skip, const void *z,
                            const float *dt_bias, const float *h0, void *y, float *h_T,
                            float *h_chunks, const int32_t *cu_seqlens, int n_seq, int B, int T,
                            int D, int G, int N, int softplus, int64_t ld_u, int64_t ld_dt,
                            int64_t ld_B, int64_t ld_C, int64_t ld_z, mdn_dtype dtype,
                            void *workspace, size_t workspace_bytes, void *stream) {
    if (D <= 0 || G <= 0 || N <= 0 || D % G || !valid_dtype(dtype) ||
        !batch_ok(cu_seqlens, n_seq, B, T))
        return MDN_ERR_INVALID_ARG;
    if (ld_u < D || ld_dt < D || (z && ld_z < D) || ld_B < (int64_t)G * N || ld_C < (int64_t)G * N)
        return MDN_ERR_INVALID_ARG;
    if (N > 128) return MDN_ERR_UNSUPPORTED;
    const long L = (long)B * T;
    const int el = element_bytes(dtype), sa = state_align(N);
    const bool some = L > 0;
    if (some && n_seq == 0) return MDN_ERR_INVALID_ARG;
    if (!Args().in(u, el, some).in(dt, el, some).in(A, sa, some).in(Bm, el, some)
             .in(Cm, el, some).in(D_skip, 4, false).in(z, el, false).in(dt_bias, 4, false)
             .in(h0, sa, false).out(y, el, some).out(h_T, sa, false, h0).out(h_chunks, 16, false).ok())
        return MDN_ERR_INVALID_ARG;
    if (some && !workspace_ok(workspace, workspace_bytes,
                              mdn_ssm_scan_fwd_workspace_size(n_seq, (int)L, D, G, N, dtype)))
        return MDN_ERR_INVALID_ARG;
    int *status = nullptr;
    const mdn_status st = current_device_status(&status);
    if (st != MDN_OK) return st;
    ScanProblem p = {};
    p.u = u; p.dt = dt; p.A = A; p.Bm = Bm; p.Cm = Cm; p.D_skip = D_skip; p.z = z;
    p.dt_bias = dt_bias; p.h0 = h0; p.y = y; p.h_T = h_T; p.h_chunks = h_chunks;
    p.ld_u = ld_u; p.ld_dt = ld_dt; p.ld_B = ld_B; p.ld_C = ld_C; p.ld_z = ld_z;
    p.cu = some ? cu_seqlens : nullptr; p.n_seq = n_seq; p.T = T; p.T_total = (int)L;
    p.D = D; p.G = G; p.N = N; p.softplus = softplus != 0;
    p.bc_wide = bc_wide(Bm, Cm, ld_B, ld_C, N, el);
    p.dtype = dtype; p.status = status;
    p.ws = static_cast<unsigned char *>(workspace);
    return finish(launch_scan_fwd(p, static_cast<cudaStream_t>(stream)));
}

mdn_status mdn_ssm_scan_bwd(const void *u, const void *dt, const float *A, const void *Bm,
                            const void *Cm, const float *D_skip, const void *z,
                            const float *dt_bias, const float *h_chunks, const void *dy,
                            const float *dh_T, void *du, void *ddt, float *dA, void *dB, void *dC,
                            float *dD_skip, void *dz, float *ddt_bias, float *dh0,
                            const int32_t *cu_seqlens, int n_seq, int B, int T, int D, int G,
                            int N, int softplus, int64_t ld_u, int64_t ld_dt, int64_t ld_B,
                            int64_t ld_C, int64_t ld_z, int64_t ld_dy, mdn_dtype dtype,
                            void *workspace, size_t workspace_bytes, void *stream) {
    if (D <= 0 || G <= 0 || N <= 0 || D % G || !valid_dtype(dtype) ||
        !batch_ok(cu_seqlens, n_seq, B, T))
        return MDN_ERR_INVALID_ARG;
    if (ld_u < D || ld_dt < D || (z && ld_z < D) || ld_dy < D || ld_B < (int64_t)G * N ||
        ld_C < (int64_t)G * N)
        return MDN_ERR_INVALID_ARG;
    if (N > 128) return MDN_ERR_UNSUPPORTED;
    const long L = (long)B * T;
    const int el = element_bytes(dtype), sa = state_align(N);
    const bool some = L > 0;
    if (some && n_seq == 0) return MDN_ERR_INVALID_ARG;
    if (!Args().in(u, el, some).in(dt, el, some).in(A, sa, some).in(Bm, el, some)
             .in(Cm, el, some).in(D_skip, 4, false).in(z, el, false).in(dt_bias, 4, false)
             .in(h_chunks, 16, some).in(dy, el, some).in(dh_T, sa, false)
             .out(du, el, some).out(ddt, el, some).out(dA, sa).out(dB, el, some).out(dC, el, some)
             .out(dD_skip, 4, false).out(dz, el, some && z).out(ddt_bias, 4, false)
             .out(dh0, sa, false).ok())
        return MDN_ERR_INVALID_ARG;
    if (some && !workspace_ok(workspace, workspace_bytes,
                              mdn_ssm_scan_bwd_workspace_size(n_seq, (int)L, D, G, N, dtype)))
        return MDN_ERR_INVALID_ARG;
    int *status = nullptr;
    const mdn_status st = current_device_status(&status);
    if (st != MDN_OK) return st;
    ScanProblem p = {};
    p.u = u; p.dt = dt; p.A = A; p.Bm = Bm; p.Cm = Cm; p.D_skip = D_skip; p.z = z;
    p.dt_bias = dt_bias; p.dy = dy; p.dh_T = dh_T;
    p.h_chunks = const_cast<float *>(h_chunks);
    p.du = du; p.ddt = ddt; p.dA = dA; p.dB = dB; p.dC = dC; p.dD = dD_skip; p.dz = dz;
    p.ddt_bias = ddt_bias; p.dh0 = dh0;
    p.ld_u = ld_u; p.ld_dt = ld_dt; p.ld_B = ld_B; p.ld_C = ld_C; p.ld_z = ld_z; p.ld_dy = ld_dy;
    p.cu = some ? cu_seqlens : nullptr; p.n_seq = n_seq; p.T = T; p.T_total = (int)L;
    p.D = D; p.G = G; p.N = N; p.softplus = softplus != 0;
    p.bc_wide = bc_wide(Bm, Cm, ld_B, ld_C, N, el);
    p.dtype = dtype; p.status = status;
    p.ws = static_cast<unsigned char *>(workspace);
    return finish(launch_scan_bwd(p, static_cast<cudaStream_t>(stream)));
}

mdn_status mdn_ssm_scan_step(const void *u, const void *dt, const float *A, const void *Bm,
                             const void *Cm, const float *D_skip, const void *z,
                             const float *dt_bias, const float *h, float *h_out, void *y, int n,
                             int D, int G, int N, int softplus, int64_t ld_u, int64_t ld_dt,
                             int64_t ld_B, int64_t ld_C, int64_t ld_z, mdn_dtype dtype,
                             void *stream) {
    if (n < 0 || D <= 0 || G <= 0 || N <= 0 || D % G || !valid_dtype(dtype))
        return MDN_ERR_INVALID_ARG;
    if (ld_u < D || ld_dt < D || (z && ld_z < D) || ld_B < (int64_t)G * N || ld_C < (int64_t)G * N)
        return MDN_ERR_INVALID_ARG;
    if (N > 128) return MDN_ERR_UNSUPPORTED;
    const int el = element_bytes(dtype), sa = state_align(N);
    const bool some = n > 0;
    if (!Args().in(u, el, some).in(dt, el, some).in(A, sa, some).in(Bm, el, some)
             .in(Cm, el, some).in(D_skip, 4, false).in(z, el, false).in(dt_bias, 4, false)
             .in(h, sa, some).out(h_out, sa, some, h).out(y, el, some).ok())
        return MDN_ERR_INVALID_ARG;
    int *status = nullptr;
    const mdn_status st = current_device_status(&status);
    if (st != MDN_OK) return st;
    ScanProblem p = {};
    p.u = u; p.dt = dt; p.A = A; p.Bm = Bm; p.Cm = Cm; p.D_skip = D_skip; p.z = z;
    p.dt_bias = dt_bias; p.h0 = h; p.h_T = h_out; p.y = y;
    p.ld_u = ld_u; p.ld_dt = ld_dt; p.ld_B = ld_B; p.ld_C = ld_C; p.ld_z = ld_z;
    p.n_seq = n; p.T = 1; p.T_total = n; p.D = D; p.G = G; p.N = N; p.softplus = softplus != 0;
    p.bc_wide = bc_wide(Bm, Cm, ld_B, ld_C, N, el);
    p.dtype = dtype; p.status = status;
    return finish(launch_scan_step(p, static_cast<cudaStream_t>(stream)));
}

static bool norm_args_ok(int rows, int D, mdn_gate_act act, float eps, mdn_dtype dtype) {
    return rows >= 0 && D > 0 && valid_dtype(dtype) && eps >= 0.f &&     // also rejects NaN
           (act == MDN_GATE_SIGMOID || act == MDN_GATE_SILU);
}

mdn_status mdn_norm_residual_fwd(const void *y, const void *x, const void *gate,
                                 const float *w_post, const float *w_pre, const float *scale,
                                 void *x_out, void *h, float *stats, int rows, int D,
                                 mdn_gate_act act, float eps, int64_t ld_y, int64_t ld_x,
                                 int64_t ld_gate, mdn_dtype dtype, void *stream) {
    if (!norm_args_ok(rows, D, act, eps, dtype) || ld_y < D || ld_x < D || (gate && ld_gate < D))
        return MDN_ERR_INVALID_ARG;
    if (D > 16384) return MDN_ERR_UNSUPPORTED;
    const int el = element_bytes(dtype);
    const bool some = rows > 0;
    if (!Args().in(y, el, some).in(x, el, some).in(gate, el, false).in(w_post, 4, false)
             .in(w_pre, 4, false).in(scale, 4, false)
             .out(x_out, el, some, ld_x == D ? x : nullptr).out(h, el, some && w_pre)
             .out(stats, 8, false).ok())
        return MDN_ERR_INVALID_ARG;
    int *status = nullptr;
    const mdn_status st = current_device_status(&status);
    if (st != MDN_OK) return st;
    NormProblem p = {};
    p.y = y; p.x = x; p.gate = gate; p.w_post = w_post; p.w_pre = w_pre; p.scale = scale;
    p.x_out = x_out; p.h = h; p.stats = stats; p.rows = rows; p.D = D; p.gate_act = act;
    p.eps = eps; p.ld_y = ld_y; p.ld_x = ld_x; p.ld_gate = ld_gate; p.dtype = dtype;
    return finish(launch_norm_fwd(p, static_cast<cudaStream_t>(stream)));
}

size_t mdn_norm_residual_bwd_workspace_size(int rows, int D, mdn_dtype dtype) {
    if (rows < 0 || D <= 0 || D > 16384 || !valid_dtype(dtype)) return 0;
    return norm_bwd_workspace(rows, D, dtype);
}

mdn_status mdn_norm_residual_bwd(const void *y, const void *x, const void *gate,
                                 const float *w_post, const float *w_pre, const float *scale,
                                 const float *stats, const void *dx_out, const void *dh, void *dy,
                                 void *dx, void *dgate, float *dw_post, float *dw_pre,
                                 float *dscale, int rows, int D, mdn_gate_act act, int64_t ld_y,
                                 int64_t ld_x, int64_t ld_gate, int64_t ld_dx_out, int64_t ld_dh,
                                 mdn_dtype dtype, void *workspace, size_t workspace_bytes,
                                 void *stream) {
    if (!norm_args_ok(rows, D, act, 0.f, dtype) || ld_y < D || ld_x < D || (gate && ld_gate < D) ||
        ld_dx_out < D || (w_pre && ld_dh < D))
        return MDN_ERR_INVALID_ARG;
    if (D > 16384) return MDN_ERR_UNSUPPORTED;
    const int el = element_bytes(dtype);
    const bool some = rows > 0;
    if (!Args().in(y, el, some).in(x, el, some).in(gate, el, false).in(w_post, 4, false)
             .in(w_pre, 4, false).in(scale, 4, false).in(stats, 8, some).in(dx_out, el, some)
             .in(dh, el, some && w_pre).out(dy, el, some)
             .out(dx, el, some, ld_dx_out == D ? dx_out : nullptr).out(dgate, el, some && gate)
             .out(dw_post, 4, w_post != nullptr).out(dw_pre, 4, w_pre != nullptr)
             .out(dscale, 4, scale != nullptr).ok())
        return MDN_ERR_INVALID_ARG;
    if (some && !workspace_ok(workspace, workspace_bytes,
                              mdn_norm_residual_bwd_workspace_size(rows, D, dtype)))
        return MDN_ERR_INVALID_ARG;
    int *status = nullptr;
    const mdn_status st = current_device_status(&status);
    if (st != MDN_OK) return st;
    NormProblem p = {};
    p.y = y; p.x = x; p.gate = gate; p.dx_out = dx_out; p.dh = dh; p.w_post = w_post;
    p.w_pre = w_pre; p.scale = scale; p.stats = const_cast<float *>(stats); p.dy = dy; p.dx = dx;
    p.dgate = dgate; p.dw_post = dw_post; p.dw_pre = dw_pre; p.dscale = dscale;
    p.partial = static_cast<float *>(workspace); p.rows = rows; p.D = D; p.gate_act = act;
    p.ld_y = ld_y; p.ld_x = ld_x; p.ld_gate = ld_gate; p.ld_dx_out = ld_dx_out; p.ld_dh = ld_dh;
    p.dtype = dtype;
    return finish(launch_norm_bwd(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
