"""Infinities in the selective scan's inputs: where the definition gives a
finite number, an infinity or NaN, so do the kernels.  Numbers of states that
fill no whole lanes, lengths that fill no whole batch of tokens and the places
behind them must not turn an infinity into NaN, or a finite number into either.
Finite values have the tolerances of ``tests/test_gpu_ssm.py``."""
import numpy as np
import pytest
import torch

from tests.test_gpu_ssm import _dev, _gen, _np, _scan_kw, _scan_ref, scan_case

pytestmark = pytest.mark.gpu

INF = float("inf")


def _same_kind(name, got, ref, mag, ulps):
    """Finite where ref is and near it, the same infinity, NaN or infinite for NaN."""
    eps = torch.finfo(got.dtype).eps / 2
    g = got.double().cpu().numpy().reshape(ref.shape)
    fin = np.isfinite(ref)
    with np.errstate(all="ignore"):
        tol = eps * np.abs(ref) + (1 + eps) * ulps * 2.0 ** -24 * np.abs(mag) + 1e-37
        tol = np.where(np.isfinite(tol), tol, np.finfo(np.float32).max)
        bad = np.where(fin, ~(np.abs(g - ref) <= tol), np.where(np.isnan(ref), np.isfinite(g), g != ref))
    at = np.argwhere(bad)
    assert not len(at), "%s: %d of %d, first at %s: %s for %s" % (name, len(at), bad.size, at[0], g[tuple(at[0])],
                                                                  ref[tuple(at[0])])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N,lens", [(16, [5, 33, 64, 1, 6, 2]), (3, [5, 33, 64, 1, 6, 2]), (20, [7, 31, 4]), (128, [9, 2]),
                                    (16, [1501]), (8, [1403, 30])])
def test_states_that_decay_at_once(dtype, N, lens):
    # A = -inf: exp(delta A) = 0 for every step, as of a very negative A
    import momentum_delta_rule_gb300 as mdn
    c = scan_case(dtype, lens, D=24, N=N, seed=N)
    c["A"][::2, ::3] = -1e30
    ref, mag = _scan_ref(c), _scan_ref(c, magnitude=True)
    d = _dev(c)
    dy, dhT = torch.randn(1, sum(lens), 24, generator=_gen(1)).to(d["u"].dtype).cuda(), torch.ones_like(d["h0"])

    def run():
        args = (d["u"], d["dt"], d["A"], d["Bm"], d["Cm"])
        y, hT, hc = mdn.ssm_scan_fwd(*args, h0=d["h0"], return_chunk_states=True, **_scan_kw(d))
        slots = sum((n + 31) // 32 for n in lens)
        g = mdn.ssm_scan_bwd(*args, hc, dy, dh_T=dhT, need_dh0=True, **_scan_kw(d))
        h = d["h0"].clone()
        n = len(lens)
        kw = {k: d[k] for k in ("D_skip", "dt_bias", "softplus")}
        ys = mdn.ssm_scan_step(d["u"][0, :n], d["dt"][0, :n], d["A"], d["Bm"][0, :n], d["Cm"][0, :n], h, **kw)
        return [y, hT, hc[:slots], ys, h] + [v for v in g.values() if v is not None]

    want = run()
    _same_kind("y", want[0], ref[0], mag[0], 64 + 16 * max(lens))
    _same_kind("h_T", want[1], ref[1], mag[1], 64 + 16 * max(lens))
    d["A"][::2, ::3] = -INF
    got = run()
    assert all(torch.isfinite(t).all() for t in want)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
