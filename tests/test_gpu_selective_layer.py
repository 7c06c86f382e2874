"""The example's stack of selective layers: the operators together, as a user
runs them.  Its prompts against an fp64 evaluation with autograd of the same
layers, its gradients against that, its single tokens against its prompts."""
import importlib.util
import os

import pytest
import torch
import torch.nn.functional as F

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("selective_layer", os.path.join(ROOT, "examples", "selective_layer.py"))
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
        for layer, p in zip(stack.layers, ps):
            xz = h @ p["w_in"]
            u, z = xz[:, :layer.inner], xz[:, layer.inner:]
            pad = F.pad(u, (0, 0, layer.width - 1, 0))
            u = F.silu((pad.unfold(0, layer.width, 1) * p["conv_w"]).sum(-1) + p["conv_b"])
            px = u @ p["w_x"]
            dt = F.softplus(px[:, :layer.rank] @ p["w_dt"] + p["dt_bias"], threshold=40.0)
            gn, rep = layer.groups * layer.n_state, layer.inner // layer.groups
            Bm, Cm = (px[:, layer.rank + i * gn:layer.rank + (i + 1) * gn]
                      .unflatten(-1, (layer.groups, layer.n_state)).repeat_interleave(rep, 1) for i in (0, 1))
            state, ys = torch.zeros(layer.inner, layer.n_state, dtype=torch.float64), []
            for t in range(len(xs)):
                state = torch.exp(dt[t, :, None] * p["A"]) * state + (dt[t] * u[t])[:, None] * Bm[t]
                ys.append((state * Cm[t]).sum(-1))
            y = (torch.stack(ys) + p["D_skip"] * u) * F.silu(z)
            res = res + p["scale"] * _rms(y @ p["w_out"], p["w_post"])
            h = _rms(res, p["w_pre"])
        out.append(h)
    return torch.cat(out)


def test_stack_and_its_gradient_against_fp64():
    ex = _example()
    # full fp32 products: TF32 would be the largest error by far
    assert not torch.backends.cuda.matmul.allow_tf32
    stack = ex.Stack(2, 24, 40, n_state=5, groups=2, dtype=torch.float32, seed=5)
    lens = [17, 3, 40]
    x = torch.randn(sum(lens), 24, generator=torch.Generator().manual_seed(1))
    cu = torch.tensor([0, 17, 20, 60], dtype=torch.int32, device="cuda")
    saves = []
    h = stack.prompt(x.cuda()[None], cu_seqlens=cu, saves=saves)
    dh = torch.randn(h.shape, generator=torch.Generator().manual_seed(2))
    dx, grads = stack.gradient(saves, dh.cuda())
    ps = [{k: v.double().cpu().requires_grad_(True) for k, v in layer.p.items()} for layer in stack.layers]
    first, x64 = stack.first.double().cpu().requires_grad_(True), x.double().requires_grad_(True)
    want = _reference(stack, ps, first, x64, lens)
    (want * dh[0].double()).sum().backward()
    # fp32 through two layers: about 1e3 roundings of 2^-24 one after another
    rel = lambda a, b: float((a.double().cpu().reshape(b.shape) - b).norm() / b.norm())
    assert rel(h, want.detach()) <= 1e-4
    assert rel(dx, x64.grad) <= 1e-4
    for g, p in zip(grads, ps):
        for k, v in p.items():
            assert rel(g[k], v.grad) <= 1e-4, k
    assert rel(grads[-1]["first"], first.grad) <= 1e-4


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-4), (torch.bfloat16, 5e-2)])
def test_tokens_continue_prompts(dtype, tol):
    ex = _example()
    stack = ex.Stack(2, 64, 128, dtype=dtype, seed=3)
    x = torch.randn(3, 50, 64, generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
    whole = stack.prompt(x)
    states = stack.new_states(3)
    head = stack.prompt(x[:, :45].contiguous(), states=states)
    rel = lambda a, b: float((a.float() - b.float()).norm() / b.float().norm())
    assert rel(head, whole[:, :45]) <= tol
    for t in range(45, 50):
        assert rel(stack.token(x[:, t].contiguous(), states), whole[:, t]) <= tol


def test_example_trains(capsys, monkeypatch):
    ex = _example()
    monkeypatch.setattr("sys.argv", ["selective_layer.py", "--steps", "16"])
    ex.main()
    losses = [float(line.split()[-1]) for line in capsys.readouterr().out.splitlines() if line.startswith("step")]
    assert len(losses) >= 3 and losses[-1] < 0.9 * losses[0]
