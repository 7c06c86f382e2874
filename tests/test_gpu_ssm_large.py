"""The state-space layer's operators on arrays whose offsets pass 32 bits: rows
far apart in a wide array, and more than 2^31 elements of dense rows.  The same
values from small arrays give the same bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu

T, D, N = 40, 64, 16


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("apart,first", [(56_000_000, 0), (56_000_001, 1)])
def test_rows_far_apart(apart, first):
    import momentum_delta_rule_gb300 as mdn
    wide = torch.empty(T, apart, dtype=torch.bfloat16, device="cuda")       # 2.24e9 elements
    assert (T - 1) * apart > 2 ** 31
    wide[:, :1024].normal_(generator=_gen(1))
    col = lambda i, n=D: wide[:, first + 64 * i:first + 64 * i + n]
    vec = lambda *s: torch.rand(*s, generator=_gen(2), device="cuda") + 0.5
    w, one, A = vec(D, 4), vec(D), -vec(D, N)

    def layer(rows):
        u, dt, z, dy = (rows(i)[None] for i in range(4))
        Bm, Cm = (rows(i, N).unflatten(-1, (1, N))[None] for i in (4, 5))
        out = list(mdn.short_conv_fwd(u, w, bias=one, output_final_state=True))
        out += [v for v in mdn.short_conv_bwd(u, w, dy, bias=one).values() if v is not None]
        y, hT, hc = mdn.ssm_scan_fwd(u, dt, A, Bm, Cm, D_skip=one, z=z, return_chunk_states=True)
        out += [y, hT] + [v for v in mdn.ssm_scan_bwd(u, dt, A, Bm, Cm, hc, dy, D_skip=one, z=z).values()
                          if v is not None]
        h = torch.ones(T, D, N, device="cuda")
        out += [mdn.ssm_scan_step(u[0], dt[0], A, Bm[0], Cm[0], h, D_skip=one, z=z[0]), h]
        state = torch.ones(T, 3, D, device="cuda", dtype=torch.bfloat16)
        out += [mdn.short_conv_step(u[0], w, state), state]
        kw = dict(w_post=one, w_pre=one, scale=one, gate=rows(2))
        X, hn, st = mdn.norm_residual_fwd(rows(0), rows(1), return_stats=True, **kw)
        out += [X, hn, st] + list(mdn.norm_residual_bwd(rows(0), rows(1), st, rows(3), dh=rows(6), **kw).values())
        return out

    # the same columns next to one another; as many elements of a row as keep its alignment
    near = wide[:, :first + 512 + (apart - 56_000_000)].clone()
    got = layer(col)
    want = layer(lambda i, n=D: near[:, first + 64 * i:first + 64 * i + n])
    torch.cuda.synchronize()
    assert mdn.device_status() == mdn.MDN_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def _last(t, n):
    return t[:, -n:].contiguous()


def test_dense_rows_of_more_than_2_31_elements():
    import momentum_delta_rule_gb300 as mdn
    width, tail = 32768, 64
    long = 2 ** 31 // width + 37
    L = long + tail
    cu = torch.tensor([0, long, L], dtype=torch.int32, device="cuda")
    x = torch.empty(1, L, width, dtype=torch.bfloat16, device="cuda").normal_(generator=_gen(3))
    vec = lambda *s: torch.rand(*s, generator=_gen(4), device="cuda") + 0.5
    w, one, A = vec(width, 4), vec(width), -vec(width, 1)
    bc = torch.ones(1, L, 1, 1, dtype=torch.bfloat16, device="cuda")
    near = _last(x, tail)

    y = mdn.short_conv_fwd(x, w, cu_seqlens=cu)[0]
    assert torch.equal(_last(y, tail), mdn.short_conv_fwd(near, w)[0])
    g = mdn.short_conv_bwd(x, w, x, cu_seqlens=cu)["dx"]
    assert torch.equal(_last(g, tail), mdn.short_conv_bwd(near, w, near)["dx"])
    del y, g

    def scan(v, cu):
        b = bc[:, :v.shape[1]]
        y, _, hc = mdn.ssm_scan_fwd(v, v, A, b, b, D_skip=one, cu_seqlens=cu, return_chunk_states=True)
        g = mdn.ssm_scan_bwd(v, v, A, b, b, hc, v, D_skip=one, cu_seqlens=cu)
        return [y, g["du"], g["ddt"]]

    two = torch.tensor([0, tail], dtype=torch.int32, device="cuda")
    for a, b in zip(scan(x, cu), scan(near, two)):
        assert torch.equal(_last(a, tail), b)

    # rows of the norms' widest
    X = x.view(1, 2 * L, width // 2)
    small = X[:, -tail:].contiguous()
    half = one[:width // 2]

    def norm(v):
        o, h, st = mdn.norm_residual_fwd(v, v, w_post=half, w_pre=half, return_stats=True)
        g = mdn.norm_residual_bwd(v, v, st, v, dh=v, w_post=half, w_pre=half)
        return [o, h, st, g["dy"], g["dx"]]

    # the forward's sums go over more threads for few rows: 2^-20 of the row's size, and bf16's step
    for k, (a, b) in enumerate(zip(norm(X), norm(small))):
        tol = 2.0 ** -20 if k == 2 else 2.0 ** -7
        assert (_last(a, tail).float() - b.float()).abs().max() <= tol * b.float().abs().max()
    torch.cuda.synchronize()
    assert mdn.device_status() == mdn.MDN_OK
