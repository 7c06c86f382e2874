"""A stack of selective state-space layers on the library's operators: prompts,
single tokens and a training step.

One layer, between the residual stream x and its normed copy h:

    u, z   = halves of h W_in
    u      = SiLU(short convolution of u)                 short_conv_*
    dt     = (u W_x)[:rank] W_dt;  B, C = the rest of u W_x
    y      = selective scan of u with dt, A, B, C, gated by z   ssm_scan_*
    x, h   = x + scale * norm(y W_out), norm of that      norm_residual_*

The projections are plain matrix products (torch).  Gradients are chained by
hand from the operators' own.

    python examples/selective_layer.py [--steps 20] [--dtype bf16]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import momentum_delta_rule_gb300 as mdn  # noqa: E402


class Layer:
    """Weights of one layer; matrices in `dtype`, the operators' parameters fp32."""

    def __init__(self, d_model, inner, n_state=16, groups=1, rank=None, width=4,
                 dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        rank = rank or math.ceil(d_model / 16)
        self.inner, self.n_state, self.groups, self.rank, self.width = inner, n_state, groups, rank, width

        def mat(a, b):
            return (torch.randn(a, b, generator=g, device=device) / math.sqrt(a)).to(dtype)

        size = torch.exp(torch.rand(inner, generator=g, device=device) * math.log(100.0) + math.log(1e-3))
        self.p = {
            "w_in": mat(d_model, 2 * inner), "w_x": mat(inner, rank + 2 * groups * n_state),
            "w_dt": mat(rank, inner), "w_out": mat(inner, d_model),
            "conv_w": torch.randn(inner, width, generator=g, device=device) / math.sqrt(width),
            "conv_b": torch.zeros(inner, device=device),
            "A": -torch.arange(1, n_state + 1, device=device, dtype=torch.float32).repeat(inner, 1),
            "D_skip": torch.ones(inner, device=device),
            "dt_bias": size + torch.log(-torch.expm1(-size)),    # softplus of it is `size`
            "scale": torch.full((d_model,), 0.5, device=device),
            "w_post": torch.ones(d_model, device=device), "w_pre": torch.ones(d_model, device=device),
        }

    def new_state(self, n, device="cuda"):
        dtype = self.p["w_in"].dtype
        return {"conv": torch.zeros(n, self.width - 1, self.inner, dtype=dtype, device=device),
                "ssm": torch.zeros(n, self.inner, self.n_state, device=device)}

    def _project(self, u):
        """dt, B, C of the convolved inputs u [..., inner]."""
        p, gn = self.p, self.groups * self.n_state
        px = u @ p["w_x"]
        dt = px[..., :self.rank] @ p["w_dt"]
        Bm, Cm = (px[..., self.rank + i * gn:self.rank + (i + 1) * gn].unflatten(-1, (self.groups, self.n_state))
                  for i in (0, 1))
        return px, dt, Bm, Cm

    def _scan_kw(self, z):
        p = self.p
        return dict(D_skip=p["D_skip"], dt_bias=p["dt_bias"], z=z)

    def _norm_kw(self):
        p = self.p
        return dict(w_post=p["w_post"], w_pre=p["w_pre"], scale=p["scale"])

    def prompt(self, x, h, cu_seqlens=None, state=None, save=None):
        """x, h [B, T, d_model] (or packed); returns x, h and fills `state` (a
        dict) with the final states.  `save` (a dict) receives what the gradient
        needs."""
        p = self.p
        xz = h @ p["w_in"]
        u0, z = xz[..., :self.inner], xz[..., self.inner:]
        conv0, ssm0 = (None, None) if state is None else (state.get("conv"), state.get("ssm"))
        u, conv_T = mdn.short_conv_fwd(u0, p["conv_w"], bias=p["conv_b"], state=conv0, cu_seqlens=cu_seqlens,
                                       output_final_state=state is not None)
        px, dt, Bm, Cm = self._project(u)
        out = mdn.ssm_scan_fwd(u, dt, p["A"], Bm, Cm, h0=ssm0, cu_seqlens=cu_seqlens,
                               output_final_state=state is not None, return_chunk_states=save is not None,
                               **self._scan_kw(z))
        y = out[0]
        o = y @ p["w_out"]
        new = mdn.norm_residual_fwd(o, x, return_stats=save is not None, **self._norm_kw())
        if state is not None:
            state.update(conv=conv_T, ssm=out[1])
        if save is not None:
            save.update(x=x, h=h, xz=xz, u=u, px=px, dt=dt, Bm=Bm, Cm=Cm, chunks=out[2], y=y, o=o, stats=new[2],
                        conv0=conv0, cu=cu_seqlens)
        return new[0], new[1]

    def token(self, x, h, state):
        """x, h [N, d_model]: one token of each sequence; `state` is updated in place."""
        p = self.p
        xz = h @ p["w_in"]
        u0, z = xz[:, :self.inner], xz[:, self.inner:]
        u = mdn.short_conv_step(u0, p["conv_w"], state["conv"], bias=p["conv_b"])
        _, dt, Bm, Cm = self._project(u)
        y = mdn.ssm_scan_step(u, dt, p["A"], Bm, Cm, state["ssm"], **self._scan_kw(z))
        return mdn.norm_residual_fwd(y @ p["w_out"], x, **self._norm_kw())

    def gradient(self, s, dx, dh):
        """Adjoints of `prompt`'s results to those of its inputs (dx, dh), and the
        weights' gradients."""
        p, g = self.p, {}
        flat = lambda t: t.flatten(0, -2)
        n = mdn.norm_residual_bwd(s["o"], s["x"], s["stats"], dx, dh=dh, **self._norm_kw())
        g.update(w_post=n["dw_post"], w_pre=n["dw_pre"], scale=n["dscale"])
        g["w_out"] = flat(s["y"]).T @ flat(n["dy"])
        z = s["xz"][..., self.inner:]
        k = mdn.ssm_scan_bwd(s["u"], s["dt"], p["A"], s["Bm"], s["Cm"], s["chunks"], n["dy"] @ p["w_out"].T,
                             cu_seqlens=s["cu"], **self._scan_kw(z))
        g.update(A=k["dA"], D_skip=k["dD_skip"], dt_bias=k["ddt_bias"])
        g["w_dt"] = flat(s["px"][..., :self.rank]).T @ flat(k["ddt"])
        dpx = torch.cat([k["ddt"] @ p["w_dt"].T, k["dB"].flatten(-2), k["dC"].flatten(-2)], -1)
        g["w_x"] = flat(s["u"]).T @ flat(dpx)
        du = k["du"] + dpx @ p["w_x"].T
        c = mdn.short_conv_bwd(s["xz"][..., :self.inner], p["conv_w"], du, bias=p["conv_b"], state=s["conv0"],
                               need_dstate=False, cu_seqlens=s["cu"])
        g.update(conv_w=c["dw"], conv_b=c["dbias"])
        dxz = torch.cat([c["dx"], k["dz"]], -1)
        g["w_in"] = flat(s["h"]).T @ flat(dxz)
        return n["dx"], dxz @ p["w_in"].T, g


class Stack:
    def __init__(self, n_layers, d_model, inner, **kw):
        seed = kw.pop("seed", 0)
        self.layers = [Layer(d_model, inner, seed=seed + i, **kw) for i in range(n_layers)]
        self.first = torch.ones(d_model, device=kw.get("device", "cuda"))

    def _enter(self, x, **kw):
        # the norm before the first block: the residual is x alone
        return mdn.norm_residual_fwd(x, torch.zeros_like(x), w_pre=self.first, **kw)

    def prompt(self, x, cu_seqlens=None, states=None, saves=None):
        entered = self._enter(x, return_stats=saves is not None)
        x0, (x, h) = x, entered[:2]
        if saves is not None:
            saves.append(dict(x0=x0, stats=entered[2]))
        for i, layer in enumerate(self.layers):
            save = None
            if saves is not None:
                save = {}
                saves.append(save)
            x, h = layer.prompt(x, h, cu_seqlens, None if states is None else states[i], save)
        return h

    def token(self, x, states):
        x, h = self._enter(x)[:2]
        for layer, state in zip(self.layers, states):
            x, h = layer.token(x, h, state)
        return h

    def gradient(self, saves, dh):
        """From the adjoint of `prompt`'s result: that of its input, and the layers'
        weight gradients (first layer first; `first` as the last entry)."""
        dx, grads = torch.zeros_like(dh), []
        for layer, s in zip(reversed(self.layers), reversed(saves[1:])):
            dx, dh, g = layer.gradient(s, dx, dh)
            grads.append(g)
        s = saves[0]
        n = mdn.norm_residual_bwd(s["x0"], torch.zeros_like(s["x0"]), s["stats"], dx, dh=dh, w_pre=self.first)
        return n["dy"], grads[::-1] + [{"first": n["dw_pre"]}]

    def new_states(self, n):
        return [layer.new_state(n) for layer in self.layers]


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--dtype", choices=["bf16", "fp32"], default="bf16")
    a = ap.parse_args()
    dtype = torch.bfloat16 if a.dtype == "bf16" else torch.float32
    torch.manual_seed(0)
    d_model, B, T = 256, 4, 200
    stack = Stack(2, d_model, 512, dtype=dtype)

    # prompts of several lengths at once, then eight more tokens of each
    lens = [70, 1, 129]
    cu = torch.tensor([0, 70, 71, 200], dtype=torch.int32, device="cuda")
    x = torch.randn(1, sum(lens), d_model, device="cuda").to(dtype)
    states = stack.new_states(len(lens))
    stack.prompt(x, cu_seqlens=cu, states=states)
    for _ in range(8):
        h = stack.token(torch.randn(len(lens), d_model, device="cuda").to(dtype), states)
    print("after %d prompt tokens and 8 steps: |h| %.3f" % (sum(lens), h.float().norm()))

    # training: the output of each position predicts the input three tokens back
    x = torch.randn(B, T, d_model, device="cuda").to(dtype)
    want = torch.nn.functional.pad(x, (0, 0, 3, 0))[:, :T].float()
    for step in range(a.steps):
        saves = []
        err = stack.prompt(x, saves=saves).float() - want
        _, grads = stack.gradient(saves, (2.0 / err.numel() * err).to(dtype))
        for layer, g in zip(stack.layers, grads):
            for k, v in layer.p.items():
                v -= (30.0 * g[k]).to(v.dtype)
        if step % 5 == 0 or step == a.steps - 1:
            print("step %2d: loss %.4f" % (step, err.square().mean()))
    assert mdn.device_status() == mdn.MDN_OK


if __name__ == "__main__":
    main()
