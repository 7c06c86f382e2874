// C ABI of linear attention with a decay for each head and of the group norm:
// argument validation and dispatch.  Declarations and the contract: include/mdn.h.
#include "mdn_args.cuh"
#include "mdn_attn.cuh"

namespace mdn {
namespace {

struct Heads {
    int n_seq;
    long L;
    int H, Hkv, dk, dv;
};

bool heads_ok(int H, int Hkv, int dk, int dv) { return H > 0 && Hkv > 0 && H % Hkv == 0 && dk > 0 && dv > 0; }
// What a call indexes with 32 bits: blocks, and channels of a token.
bool heads_small(long n_seq, long L, int H, int dk, int dv) {
    const long seg_slots = n_seq + L / 64;
    return dk <= 128 && dv <= 128 && (long)H * 128 <= 0x7fffffffL && seg_slots * H <= 0x7fffffffL;
}

// The workspace: packed sequences' items, the segments' states (fp32) and, for
// shared heads, their gradients by query head (fp32).
struct Space {
    size_t items = 0, offs = 0, states = 0, states2 = 0, dk = 0, dv = 0, total = 0;
    int seg = 0;
    long slots = 0;
};
Space space(const Heads &s, bool packed, mdn_dtype dtype, bool bwd) {
    Space w;
    if (s.L == 0) return w;
    w.seg = attn_segment(s.n_seq, s.L, s.H, bwd ? 3 : 1, dtype);
    w.slots = attn_slots(s.n_seq, s.L, w.seg);
    auto take = [&](size_t bytes) {
        const size_t at = w.total;
        w.total += round256(bytes);
        return at;
    };
    w.items = take(packed ? w.slots * sizeof(AttnItem) : 0);
    w.offs = take(packed ? (s.n_seq + 2) * sizeof(int32_t) : 0);
    const size_t states = w.seg ? (size_t)w.slots * s.H * s.dk * s.dv * sizeof(float) : 0;
    w.states = take(states);
    if (bwd) {
        w.states2 = take(states);
        const bool shared = s.H != s.Hkv;
        w.dk = take(shared ? (size_t)s.L * s.H * s.dk * sizeof(float) : 0);
        w.dv = take(shared ? (size_t)s.L * s.H * s.dv * sizeof(float) : 0);
    }
    return w;
}

// Whether a kernel of its own joins the segments' states, rather than each block
// those before its own: blocks read a state in 2.5 us, the kernel takes 8 and its
// launch 2.  (16 heads of 128 over 16384 tokens in 9 segments: 118 us and 108; 64
// over 2048 tokens in 2: 64 and 69.)
bool many_segments(const Space &w, int n_seq, long L) { return L / n_seq > 3L * w.seg; }

AttnProblem problem(const Heads &s, const Space &w, const float *log_decay, const int32_t *cu, int T, mdn_dtype dtype,
                    int *status, unsigned char *ws) {
    AttnProblem p = {};
    p.log_decay = log_decay;
    p.H = s.H;
    p.n_seq = s.n_seq;
    p.T = T;
    p.T_total = (int)s.L;
    p.seg = w.seg;
    p.cu = cu;
    p.dtype = dtype;
    p.status = status;
    if (p.cu) {
        p.slots = (int)w.slots;
        // (few whole sequences order themselves)
        if (w.seg || s.n_seq > kAttnOrdered) p.items = reinterpret_cast<AttnItem *>(ws + w.items);
        p.seg_off = reinterpret_cast<int32_t *>(ws + w.offs);
    } else {
        p.slots = s.n_seq * (w.seg ? (T + w.seg - 1) / w.seg : 1);
    }
    return p;
}

// Without tokens the states stay as they are: no kernel, which would read the
// decays that such a call need not have.
cudaError_t keep_states(const Heads &s, float *to, const float *from, cudaStream_t st) {
    const size_t bytes = (size_t)s.n_seq * s.H * s.dk * s.dv * sizeof(float);
    if (to == nullptr || to == from || bytes == 0) return cudaSuccess;
    return from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, st) : cudaMemsetAsync(to, 0, bytes, st);
}

}  // namespace
}  // namespace mdn

using namespace mdn;

extern "C" {

static size_t attn_workspace(int n_seq, int T_total, int H, int Hkv, int dk, int dv, int packed, mdn_dtype dtype, bool bwd) {
    if (n_seq < 0 || T_total < 0 || !heads_ok(H, Hkv, dk, dv) || !valid_dtype(dtype) ||
        !heads_small(n_seq, T_total, H, dk, dv))
        return 0;
    return space(Heads{n_seq, T_total, H, Hkv, dk, dv}, packed != 0, dtype, bwd).total;
}
size_t mdn_linear_attn_fwd_workspace_size(int n_seq, int T_total, int H, int Hkv, int dk, int dv, int packed,
                                          mdn_dtype dtype) {
    return attn_workspace(n_seq, T_total, H, Hkv, dk, dv, packed, dtype, false);
}
size_t mdn_linear_attn_bwd_workspace_size(int n_seq, int T_total, int H, int Hkv, int dk, int dv, int packed,
                                          mdn_dtype dtype) {
    return attn_workspace(n_seq, T_total, H, Hkv, dk, dv, packed, dtype, true);
}

mdn_status mdn_linear_attn_fwd(const void *q, const void *k, const void *v, const float *log_decay, const float *S0,
                               void *o, float *S_T, const int32_t *cu_seqlens, int n_seq, int B, int T, int H, int Hkv,
                               int dk, int dv, float scale, int64_t ld_q, int64_t ld_k, int64_t ld_v, mdn_dtype dtype,
                               void *workspace, size_t workspace_bytes, void *stream) {
    if (!heads_ok(H, Hkv, dk, dv) || !valid_dtype(dtype) || !batch_ok(cu_seqlens, n_seq, B, T) ||
        ld_q < (int64_t)H * dk || ld_k < (int64_t)Hkv * dk || ld_v < (int64_t)Hkv * dv)
        return MDN_ERR_INVALID_ARG;
    const long L = (long)B * T;
    if (!heads_small(n_seq, L, H, dk, dv)) return MDN_ERR_UNSUPPORTED;
    const int el = element_bytes(dtype), sa = state_align(dv);
    const bool some = L > 0;
    if (some && n_seq == 0) return MDN_ERR_INVALID_ARG;
    if (!Args().in(q, el, some).in(k, el, some).in(v, el, some).in(log_decay, 4, some).in(S0, sa, false)
             .out(o, el, some).out(S_T, sa, false, S0).ok())
        return MDN_ERR_INVALID_ARG;
    const Heads s{n_seq, L, H, Hkv, dk, dv};
    const Space w = space(s, cu_seqlens != nullptr, dtype, false);
    if (!workspace_ok(workspace, workspace_bytes, w.total)) return MDN_ERR_INVALID_ARG;
    int *status = nullptr;
    const mdn_status st = current_device_status(&status);
    if (st != MDN_OK) return st;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (!some) return finish(keep_states(s, S_T, S0, cs));
    AttnProblem p = problem(s, w, log_decay, cu_seqlens, T, dtype, status, ws);
    AttnPass a = {};
    a.X = q; a.Y = k; a.W = v;
    a.ld_x = ld_q; a.ld_y = ld_k; a.ld_w = ld_v;
    a.sx = 1; a.sy = a.sw = H / Hkv;
    a.kd = dk; a.vd = dv;
    a.out_scale = scale; a.w_scale = 1.f;
    cudaError_t err = cudaSuccess;
    if (p.items) err = launch_attn_layout(p, cs);
    if (w.seg && err == cudaSuccess) {
        a.seg_out = reinterpret_cast<float *>(ws + w.states);
        a.init = S0;
        p.pass[0] = a;
        p.n_pass = 1;
        err = launch_attn(p, cs);
        a.combined = many_segments(w, n_seq, L);
        if (a.combined && err == cudaSuccess) err = launch_attn_combine(p, a.seg_out, nullptr, dk * dv, cs);
        a.seg_init = a.seg_out;
        a.seg_out = nullptr;
    }
    a.init = S0;
    a.fin = S_T;
    a.out = o;
    p.pass[0] = a;
    p.n_pass = 1;
    if (err == cudaSuccess) err = launch_attn(p, cs);
    return finish(err);
}

mdn_status mdn_linear_attn_bwd(const void *q, const void *k, const void *v, const float *log_decay, const float *S0,
                               const void *d_o, const float *dS_T, void *dq, void *dk_out, void *dv_out, float *dS0,
                               const int32_t *cu_seqlens, int n_seq, int B, int T, int H, int Hkv, int dk, int dv,
                               float scale, int64_t ld_q, int64_t ld_k, int64_t ld_v, int64_t ld_do, mdn_dtype dtype,
                               void *workspace, size_t workspace_bytes, void *stream) {
    if (!heads_ok(H, Hkv, dk, dv) || !valid_dtype(dtype) || !batch_ok(cu_seqlens, n_seq, B, T) ||
        ld_q < (int64_t)H * dk || ld_k < (int64_t)Hkv * dk || ld_v < (int64_t)Hkv * dv || ld_do < (int64_t)H * dv)
        return MDN_ERR_INVALID_ARG;
    const long L = (long)B * T;
    if (!heads_small(n_seq, L, H, dk, dv)) return MDN_ERR_UNSUPPORTED;
    const int el = element_bytes(dtype), sa = dk % 4 == 0 || dv % 4 == 0 ? 16 : 4;
    const bool some = L > 0;
    if (some && n_seq == 0) return MDN_ERR_INVALID_ARG;
    if (!Args().in(q, el, some).in(k, el, some).in(v, el, some).in(log_decay, 4, some).in(S0, sa, false)
             .in(d_o, el, some).in(dS_T, sa, false).out(dq, el, some).out(dk_out, el, some).out(dv_out, el, some)
             .out(dS0, sa, false).ok())
        return MDN_ERR_INVALID_ARG;
    const Heads s{n_seq, L, H, Hkv, dk, dv};
    const Space w = space(s, cu_seqlens != nullptr, dtype, true);
    if (!workspace_ok(workspace, workspace_bytes, w.total)) return MDN_ERR_INVALID_ARG;
    int *status = nullptr;
    const mdn_status st = current_device_status(&status);
    if (st != MDN_OK) return st;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (!some) return finish(keep_states(s, dS0, dS_T, cs));
    AttnProblem p = problem(s, w, log_decay, cu_seqlens, T, dtype, status, ws);
    const int shared = H / Hkv;
    // the segments' own states: S, and dS at their ends
    AttnPass fwd = {}, rev = {};
    fwd.Y = k; fwd.W = v;
    fwd.ld_y = ld_k; fwd.ld_w = ld_v;
    fwd.sx = 1; fwd.sy = fwd.sw = shared;
    fwd.kd = dk; fwd.vd = dv;
    fwd.w_scale = 1.f;
    rev.Y = q; rev.W = d_o;
    rev.ld_y = ld_q; rev.ld_w = ld_do;
    rev.sx = rev.sy = rev.sw = 1;
    rev.kd = dk; rev.vd = dv;
    rev.reversed = true;
    rev.w_scale = scale;
    cudaError_t err = cudaSuccess;
    if (p.items) err = launch_attn_layout(p, cs);
    const float *seg_S = nullptr, *seg_dS = nullptr;
    bool combined = false;
    if (w.seg && err == cudaSuccess) {
        fwd.seg_out = reinterpret_cast<float *>(ws + w.states);
        fwd.init = S0;
        rev.init = dS_T;
        rev.seg_out = reinterpret_cast<float *>(ws + w.states2);
        p.pass[0] = fwd;
        p.pass[1] = rev;
        p.n_pass = 2;
        err = launch_attn(p, cs);
        combined = many_segments(w, n_seq, L);
        if (combined && err == cudaSuccess) err = launch_attn_combine(p, fwd.seg_out, rev.seg_out, dk * dv, cs);
        seg_S = fwd.seg_out;
        seg_dS = rev.seg_out;
    }
    void *to_dk = shared > 1 ? static_cast<void *>(ws + w.dk) : dk_out;
    void *to_dv = shared > 1 ? static_cast<void *>(ws + w.dv) : dv_out;
    AttnPass a = {};
    a.X = d_o; a.Y = v; a.W = k;
    a.ld_x = ld_do; a.ld_y = ld_v; a.ld_w = ld_k;
    a.sx = 1; a.sy = a.sw = shared;
    a.kd = dv; a.vd = dk;
    a.out_scale = scale; a.w_scale = 1.f;
    a.out = dq;
    a.init = S0; a.seg_init = seg_S; a.init_t = true;
    AttnPass b = {};
    b.X = v; b.Y = d_o; b.W = q;
    b.ld_x = ld_v; b.ld_y = ld_do; b.ld_w = ld_q;
    b.sx = shared; b.sy = b.sw = 1;
    b.kd = dv; b.vd = dk;
    b.reversed = true;
    b.out_scale = 1.f; b.w_scale = scale;
    b.out = to_dk; b.out_f32 = shared > 1;
    b.init = dS_T; b.seg_init = seg_dS; b.init_t = true;
    a.combined = b.combined = combined;
    AttnPass c = rev;
    c.combined = combined;
    c.seg_out = nullptr;
    c.X = k; c.ld_x = ld_k; c.sx = shared;
    c.out_scale = 1.f;
    c.out = to_dv; c.out_f32 = shared > 1;
    c.init = dS_T; c.seg_init = seg_dS;
    c.fin = dS0;
    p.pass[0] = a;
    p.pass[1] = b;
    p.pass[2] = c;
    p.n_pass = 3;
    if (err == cudaSuccess) err = launch_attn(p, cs);
    if (shared > 1) {
        if (err == cudaSuccess) err = launch_attn_reduce(p, reinterpret_cast<float *>(ws + w.dk), dk_out, dk, shared, cs);
        if (err == cudaSuccess) err = launch_attn_reduce(p, reinterpret_cast<float *>(ws + w.dv), dv_out, dv, shared, cs);
    }
    return finish(err);
}

mdn_status mdn_linear_attn_step(const void *q, const void *k, const void *v, const float *log_decay, const float *S,
                                float *S_out, void *o, int n, int H, int Hkv, int dk, int dv, float scale, int64_t ld_q,
                                int64_t ld_k, int64_t ld_v, mdn_dtype dtype, void *stream) {
    if (n < 0 || !heads_ok(H, Hkv, dk, dv) || !valid_dtype(dtype) || ld_q < (int64_t)H * dk ||
        ld_k < (int64_t)Hkv * dk || ld_v < (int64_t)Hkv * dv)
        return MDN_ERR_INVALID_ARG;
    if (!heads_small(n, 0, H, dk, dv)) return MDN_ERR_UNSUPPORTED;
    const int el = element_bytes(dtype), sa = state_align(dv);
    const bool some = n > 0;
    if (!Args().in(q, el, some).in(k, el, some).in(v, el, some).in(log_decay, 4, some).in(S, sa, some)
             .out(S_out, sa, some, S).out(o, el, some).ok())
        return MDN_ERR_INVALID_ARG;
    int *status = nullptr;
    const mdn_status st = current_device_status(&status);
    if (st != MDN_OK) return st;
    AttnStepProblem p = {};
    p.q = q; p.k = k; p.v = v; p.log_decay = log_decay; p.S = S; p.S_out = S_out; p.o = o;
    p.n = n; p.H = H; p.shared = H / Hkv; p.dk = dk; p.dv = dv; p.scale = scale;
    p.ld_q = ld_q; p.ld_k = ld_k; p.ld_v = ld_v; p.dtype = dtype;
    return finish(launch_attn_step(p, static_cast<cudaStream_t>(stream)));
}

static bool group_norm_ok(int D, int G, mdn_norm_act act, float eps, mdn_dtype dtype) {
    return D > 0 && G > 0 && D % G == 0 && valid_dtype(dtype) && eps >= 0.f &&      // also rejects NaN
           (act == MDN_ACT_NONE || act == MDN_ACT_SILU || act == MDN_ACT_SIGMOID);
}

size_t mdn_group_norm_fwd_workspace_size(int n_seq, int rows, int D, int G, int over_sequence, mdn_dtype dtype) {
    if (n_seq < 0 || rows < 0 || !group_norm_ok(D, G, MDN_ACT_NONE, 0.f, dtype) || D > 16384) return 0;
    return group_norm_fwd_workspace(n_seq, rows, D, G, over_sequence != 0, dtype);
}
size_t mdn_group_norm_bwd_workspace_size(int n_seq, int rows, int D, int G, int over_sequence, mdn_dtype dtype) {
    if (n_seq < 0 || rows < 0 || !group_norm_ok(D, G, MDN_ACT_NONE, 0.f, dtype) || D > 16384) return 0;
    return group_norm_bwd_workspace(n_seq, rows, D, G, over_sequence != 0, dtype);
}

mdn_status mdn_group_norm_fwd(const void *x, const void *gate, const float *weight, const float *bias, void *y,
                              float *stats, const int32_t *cu_seqlens, int n_seq, int B, int T, int D, int G,
                              int over_sequence, int center, mdn_norm_act act, float eps, int64_t ld_x, int64_t ld_gate,
                              mdn_dtype dtype, void *workspace, size_t workspace_bytes, void *stream) {
    if (!group_norm_ok(D, G, act, eps, dtype) || !batch_ok(cu_seqlens, n_seq, B, T) || (cu_seqlens && !over_sequence) ||
        ld_x < D || (gate && ld_gate < D))
        return MDN_ERR_INVALID_ARG;
    if (D > 16384) return MDN_ERR_UNSUPPORTED;
    const long L = (long)B * T;
    const int el = element_bytes(dtype);
    const bool some = L > 0;
    if (some && n_seq == 0) return MDN_ERR_INVALID_ARG;
    if (!Args().in(x, el, some).in(gate, el, false).in(weight, 4, false).in(bias, 4, false).out(y, el, some)
             .out(stats, 8, false).ok())
        return MDN_ERR_INVALID_ARG;
    if (some && !workspace_ok(workspace, workspace_bytes,
                              group_norm_fwd_workspace(n_seq, L, D, G, over_sequence != 0, dtype)))
        return MDN_ERR_INVALID_ARG;
    int *status = nullptr;
    const mdn_status st = current_device_status(&status);
    if (st != MDN_OK) return st;
    GroupNormProblem p = {};
    p.x = x; p.gate = gate; p.weight = weight; p.bias = bias; p.y = y; p.stats = stats;
    p.cu = some ? cu_seqlens : nullptr; p.n_seq = n_seq; p.T = T; p.rows = L; p.D = D; p.G = G; p.act = act;
    p.over_sequence = over_sequence != 0; p.center = center != 0; p.eps = eps;
    p.ld_x = ld_x; p.ld_gate = ld_gate; p.dtype = dtype;
    p.ws = static_cast<unsigned char *>(workspace); p.status = status;
    return finish(launch_group_norm_fwd(p, static_cast<cudaStream_t>(stream)));
}

mdn_status mdn_group_norm_bwd(const void *x, const void *gate, const float *weight, const float *bias,
                              const float *stats, const void *dy, void *dx, void *dgate, float *dw, float *dbias,
                              const int32_t *cu_seqlens, int n_seq, int B, int T, int D, int G, int over_sequence,
                              int center, mdn_norm_act act, int64_t ld_x, int64_t ld_gate, int64_t ld_dy,
                              mdn_dtype dtype, void *workspace, size_t workspace_bytes, void *stream) {
    if (!group_norm_ok(D, G, act, 0.f, dtype) || !batch_ok(cu_seqlens, n_seq, B, T) || (cu_seqlens && !over_sequence) ||
        ld_x < D || (gate && ld_gate < D) || ld_dy < D)
        return MDN_ERR_INVALID_ARG;
    if (D > 16384) return MDN_ERR_UNSUPPORTED;
    const long L = (long)B * T;
    const int el = element_bytes(dtype);
    const bool some = L > 0;
    if (some && n_seq == 0) return MDN_ERR_INVALID_ARG;
    if (!Args().in(x, el, some).in(gate, el, false).in(weight, 4, false).in(bias, 4, false).in(stats, 8, some)
             .in(dy, el, some).out(dx, el, some).out(dgate, el, some && gate).out(dw, 4, false).out(dbias, 4, false).ok())
        return MDN_ERR_INVALID_ARG;
    if (some && !workspace_ok(workspace, workspace_bytes,
                              group_norm_bwd_workspace(n_seq, L, D, G, over_sequence != 0, dtype)))
        return MDN_ERR_INVALID_ARG;
    int *status = nullptr;
    const mdn_status st = current_device_status(&status);
    if (st != MDN_OK) return st;
    GroupNormProblem p = {};
    p.x = x; p.gate = gate; p.weight = weight; p.bias = bias; p.stats = const_cast<float *>(stats); p.dy = dy;
    p.dx = dx; p.dgate = dgate; p.dw = dw; p.dbias = dbias;
    p.cu = some ? cu_seqlens : nullptr; p.n_seq = n_seq; p.T = T; p.rows = L; p.D = D; p.G = G; p.act = act;
    p.over_sequence = over_sequence != 0; p.center = center != 0;
    p.ld_x = ld_x; p.ld_gate = ld_gate; p.ld_dy = ld_dy; p.dtype = dtype;
    p.ws = static_cast<unsigned char *>(workspace); p.status = status;
    return finish(launch_group_norm_bwd(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
