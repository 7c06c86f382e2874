"""A stack of linear-attention layers on the library's operators: prompts, single
tokens and a training step.

One layer, between the residual stream x and its normed copy h:

    q k v, z = parts of h W_in
    q k v    = SiLU(short convolution of q k v)                short_conv_*
    o        = linear attention with a decay for each head     linear_attn_*
    y        = norm of each head's o, times SiLU(z)            group_norm_*
    x, h     = x + scale * norm(y W_out), norm of that         norm_residual_*

Several query heads may share a key and value head.  The projections are plain
matrix products (torch).  Gradients are chained by hand from the operators' own.

    python examples/linear_attention_layer.py [--steps 20] [--dtype bf16]
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

    def __init__(self, d_model, heads, dk, dv, kv_heads=None, width=4, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.H, self.Hkv, self.dk, self.dv, self.width = heads, kv_heads or heads, dk, dv, width
        self.qkv = heads * dk + self.Hkv * (dk + dv)
        self.scale = dk ** -0.5

        def mat(a, b):
            return (torch.randn(a, b, generator=g, device=device) / math.sqrt(a)).to(dtype)

        self.p = {
            "w_in": mat(d_model, self.qkv + heads * dv), "w_out": mat(heads * dv, d_model),
            "conv_w": torch.randn(self.qkv, width, generator=g, device=device) / math.sqrt(width),
            "conv_b": torch.zeros(self.qkv, device=device),
            "norm_w": torch.ones(heads * dv, device=device), "norm_b": torch.zeros(heads * dv, device=device),
            "scale": torch.full((d_model,), 0.5, device=device),
            "w_post": torch.ones(d_model, device=device), "w_pre": torch.ones(d_model, device=device),
        }
        # time constants from two tokens to 256, geometrically over the heads
        self.log_decay = -torch.exp2(-8.0 * (torch.arange(heads, device=device, dtype=torch.float32) + 1) / heads)

    def new_state(self, n, device="cuda"):
        dtype = self.p["w_in"].dtype
        return {"conv": torch.zeros(n, self.width - 1, self.qkv, dtype=dtype, device=device),
                "S": torch.zeros(n, self.H, self.dk, self.dv, device=device)}

    def _split(self, u):
        """q, k and v of the convolved projection, as heads."""
        q, k, v = u.split([self.H * self.dk, self.Hkv * self.dk, self.Hkv * self.dv], dim=-1)
        return (q.unflatten(-1, (self.H, self.dk)), k.unflatten(-1, (self.Hkv, self.dk)),
                v.unflatten(-1, (self.Hkv, self.dv)), self.log_decay)

    def _head_norm_kw(self, z):
        return dict(weight=self.p["norm_w"], bias=self.p["norm_b"], gate=z, activation="silu")

    def _norm_kw(self):
        p = self.p
        return dict(w_post=p["w_post"], w_pre=p["w_pre"], scale=p["scale"])

    def prompt(self, x, h, cu_seqlens=None, state=None, save=None):
        """x, h [B, T, d_model] (or packed); returns x, h and fills `state` (a
        dict) with the final states.  `save` (a dict) receives what the gradient
        needs."""
        p = self.p
        a = h @ p["w_in"]
        conv0, S0 = (None, None) if state is None else (state.get("conv"), state.get("S"))
        u, conv_T = mdn.short_conv_fwd(a[..., :self.qkv], p["conv_w"], bias=p["conv_b"], state=conv0, cu_seqlens=cu_seqlens,
                                       output_final_state=state is not None)
        o, S_T = mdn.linear_attn_fwd(*self._split(u), scale=self.scale, S0=S0, cu_seqlens=cu_seqlens,
                                     output_final_state=state is not None)
        y, heads = mdn.group_norm_fwd(o.flatten(-2), self.H, return_stats=True, **self._head_norm_kw(a[..., self.qkv:]))
        r = y @ p["w_out"]
        new = mdn.norm_residual_fwd(r, x, return_stats=save is not None, **self._norm_kw())
        if state is not None:
            state.update(conv=conv_T, S=S_T)
        if save is not None:
            save.update(x=x, h=h, a=a, u=u, o=o, y=y, r=r, heads=heads, stats=new[2], conv0=conv0, S0=S0, cu=cu_seqlens)
        return new[0], new[1]

    def token(self, x, h, state):
        """x, h [N, d_model]: one token of each sequence; `state` is updated in place."""
        p = self.p
        a = h @ p["w_in"]
        u = mdn.short_conv_step(a[:, :self.qkv], p["conv_w"], state["conv"], bias=p["conv_b"])
        o = mdn.linear_attn_step(*self._split(u), state["S"], scale=self.scale)
        y = mdn.group_norm_fwd(o.flatten(-2), self.H, **self._head_norm_kw(a[:, self.qkv:]))
        return mdn.norm_residual_fwd(y @ p["w_out"], x, **self._norm_kw())

    def gradient(self, s, dx, dh):
        """Adjoints of `prompt`'s results to those of its inputs (dx, dh), and the
        weights' gradients."""
        p, g = self.p, {}
        flat = lambda t: t.flatten(0, -2)
        n = mdn.norm_residual_bwd(s["r"], s["x"], s["stats"], dx, dh=dh, **self._norm_kw())
        g.update(w_post=n["dw_post"], w_pre=n["dw_pre"], scale=n["dscale"])
        g["w_out"] = flat(s["y"]).T @ flat(n["dy"])
        m = mdn.group_norm_bwd(s["o"].flatten(-2), self.H, s["heads"], n["dy"] @ p["w_out"].T,
                               **self._head_norm_kw(s["a"][..., self.qkv:]))
        g.update(norm_w=m["dw"], norm_b=m["dbias"])
        k = mdn.linear_attn_bwd(*self._split(s["u"]), m["dx"].unflatten(-1, (self.H, self.dv)), scale=self.scale, S0=s["S0"],
                                cu_seqlens=s["cu"], need_dS0=False)
        du = torch.cat([k[i].flatten(-2) for i in ("dq", "dk", "dv")], -1)
        c = mdn.short_conv_bwd(s["a"][..., :self.qkv], p["conv_w"], du, bias=p["conv_b"], state=s["conv0"], need_dstate=False,
                               cu_seqlens=s["cu"])
        g.update(conv_w=c["dw"], conv_b=c["dbias"])
        da = torch.cat([c["dx"], m["dgate"]], -1)
        g["w_in"] = flat(s["h"]).T @ flat(da)
        return n["dx"], da @ p["w_in"].T, g


class Stack:
    def __init__(self, n_layers, d_model, heads, dk, dv, **kw):
        seed = kw.pop("seed", 0)
        self.layers = [Layer(d_model, heads, dk, dv, seed=seed + i, **kw) for i in range(n_layers)]
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
    stack = Stack(2, d_model, 8, 32, 64, kv_heads=4, dtype=dtype)

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
        print("step %2d: mean squared error %.4f" % (step, err.square().mean()))
        _, grads = stack.gradient(saves, (err * (2.0 / err.numel())).to(dtype))
        for layer, g in zip(stack.layers, grads):
            for name, d in g.items():
                w = layer.p[name]
                w.sub_((d.float() * 30.0).to(w.dtype))
        stack.first.sub_(grads[-1]["first"] * 30.0)


if __name__ == "__main__":
    main()
