"""The example's stack of linear-attention layers: the operators together, as a
user runs them.  Its prompts against an fp64 evaluation with autograd of the
same layers, its gradients against that, its single tokens against its prompts."""
import importlib.util
import os

import pytest
import torch
import torch.nn.functional as F

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("linear_attention_layer",
                                                  os.path.join(ROOT, "examples", "linear_attention_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _rms(x, w):
    return x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w


def _reference(stack, ps, first, x, lens):
    """The stack in fp64 on the CPU; ps: its layers' weights."""
    out = []
    for xs in x.split(lens):
        res, h = xs, _rms(xs, first)
        n = len(xs)
        t = torch.arange(n, dtype=torch.float64)
        for layer, p in zip(stack.layers, ps):
            a = h @ p["w_in"]
            u, z = a[:, :layer.qkv], a[:, layer.qkv:]
            pad = F.pad(u, (0, 0, layer.width - 1, 0))
            u = F.silu((pad.unfold(0, layer.width, 1) * p["conv_w"]).sum(-1) + p["conv_b"])
            H, Hkv, dk, dv = layer.H, layer.Hkv, layer.dk, layer.dv
            q, k, v = u.split([H * dk, Hkv * dk, Hkv * dv], -1)
            q = q.unflatten(-1, (H, dk))
            k, v = (m.unflatten(-1, (Hkv, -1)).repeat_interleave(H // Hkv, 1) for m in (k, v))
            decay = torch.exp(layer.log_decay.double().cpu()[:, None, None] * (t[:, None] - t).clamp(min=0)).tril()
            o = torch.einsum("hij,jhv->ihv", torch.einsum("ihk,jhk->hij", q, k) * decay * layer.scale, v)
            o = (o - o.mean(-1, keepdim=True)) / (o.var(-1, unbiased=False, keepdim=True) + 1e-5).sqrt()
            y = (o.flatten(1) * p["norm_w"] + p["norm_b"]) * F.silu(z)
            res = res + p["scale"] * _rms(y @ p["w_out"], p["w_post"])
            h = _rms(res, p["w_pre"])
        out.append(h)
    return torch.cat(out)


def test_stack_and_its_gradient_against_fp64():
    ex = _example()
    # full fp32 products: TF32 would be the largest error by far
    assert not torch.backends.cuda.matmul.allow_tf32
    stack = ex.Stack(2, 24, 4, 9, 12, kv_heads=2, dtype=torch.float32, seed=5)
    lens = [17, 3, 70]
    x = torch.randn(sum(lens), 24, generator=torch.Generator().manual_seed(1))
    cu = torch.tensor([0, 17, 20, 90], dtype=torch.int32, device="cuda")
    saves = []
    h = stack.prompt(x[None].cuda(), cu_seqlens=cu, saves=saves)
    dh = torch.randn(h.shape, generator=torch.Generator().manual_seed(2))
    dx, grads = stack.gradient(saves, dh.cuda())
    torch.cuda.synchronize()

    leaf = lambda t: t.detach().double().cpu().requires_grad_()
    ps = [{k: leaf(v) for k, v in layer.p.items()} for layer in stack.layers]
    first, xr = leaf(stack.first), leaf(x)
    ref = _reference(stack, ps, first, xr, lens)
    (ref * dh[0].double()).sum().backward()
    # two layers of some ten operators, each of relative error below 1e-6 of its
    # result in norm; a norm of a head may stretch what it is given by its
    # factor, a few times
    close = lambda a, b: (a.double().cpu().reshape(b.shape) - b).norm() <= 1e-4 * b.norm()
    assert close(h, ref.detach())
    assert close(dx, xr.grad)
    for g, p in zip(grads, ps):
        assert set(g) == set(p)
        for name in g:
            assert close(g[name], p[name].grad), name
    assert close(grads[-1]["first"], first.grad)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tokens_continue_prompts(dtype):
    ex = _example()
    stack = ex.Stack(2, 64, 4, 16, 32, kv_heads=2, dtype=dtype, seed=7)
    x = torch.randn(3, 75, 64, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    want = stack.prompt(x)
    states = [{} for _ in stack.layers]
    got = [stack.prompt(x[:, :66].contiguous(), states=states)]
    for t in range(66, 75):
        got.append(stack.token(x[:, t].contiguous(), states)[:, None])
    torch.cuda.synchronize()
    off = (torch.cat(got, 1).float() - want.float()).norm() / want.float().norm()
    # bf16: the two ways round q k^T or the states differently, and everything
    # behind them by a step here and there
    assert off <= (1e-5 if dtype == torch.float32 else 3e-2), off


def test_a_step_of_the_layer_in_a_graph():
    ex = _example()
    stack = ex.Stack(2, 64, 4, 16, 32, dtype=torch.bfloat16, seed=9)
    states = stack.new_states(5)
    x = torch.randn(5, 64, device="cuda").bfloat16()
    for _ in range(2):
        stack.token(x, states)
    kept = [{k: v.clone() for k, v in s.items()} for s in states]
    want = stack.token(x, states)
    after = [{k: v.clone() for k, v in s.items()} for s in states]
    for s, k in zip(states, kept):
        for name in s:
            s[name].copy_(k[name])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = stack.token(x, states)
    for s, k in zip(states, kept):
        for name in s:
            s[name].copy_(k[name])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    for s, k in zip(states, after):
        for name in s:
            assert torch.equal(s[name], k[name])


def test_the_example_runs():
    import subprocess
    import sys
    out = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "linear_attention_layer.py"), "--steps", "2"],
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    assert "step  1" in out.stdout
