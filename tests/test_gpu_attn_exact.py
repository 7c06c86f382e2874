"""bf16 rows are a matter of the rows alone: outputs and gradients of linear
attention on bf16 rows are the formulas' on those rows, rounded to bf16 once, and
states, which are fp32, have fp32's errors.

Outputs.  Let y be what a kernel rounds to x, E a bound of |y - ref|.  Where x is
not the number that ref itself rounds to, r, the middle between the two lies
between y and ref, so that |x - ref| is at most half a step and E more, and |r -
ref| at least half a step less E.  In all cases |x - ref| <= |r - ref| + 2 E.  With
the magnitude m of a value's terms (the reference formula over absolute values)
E is
  * U m for the fp32 sums and (late - m) for the decays' exponents, as in
    test_gpu_attn.py;
  * 2^-16 m: a term passes one operand (the decayed q k^T or the state) that is
    taken as two bf16 parts, the first off by half a step, 2^-8, the second by
    half a step of that at most.

States of at most 16 tokens, which a product of one step takes at once.  In
steps of 2^-24: a decay's exp2, its products with the scale and a row and the scale
itself 7, the sum of T products and the carried state T + 1, each addition cut
short rather than rounded (twice as much), three parts of 8 bits each leave 1,
the decayed initial state 5 and its sum 1: (2 T + 16) 2^-24 m, beside (late - m).
"""
import numpy as np
import pytest
import torch

from tests.test_gpu_attn import case, dev, flat, reference, run

pytestmark = pytest.mark.gpu


def bounds(c, steps, parts):
    ref, mag = flat(reference(c)), flat(reference(c, magnitude=True))
    late = flat(reference(c, magnitude=True, exponent_error=4 * 2.0 ** -24))
    return ref, {n: (steps * 2.0 ** -24 + parts) * mag[n] + (late[n] - mag[n]) + 1e-37 for n in ref}


def check_rounded_once(c, got):
    T, (dk, dv) = max(c["lens"]), (c["q"].shape[-1], c["v"].shape[-1])
    ref, E = bounds(c, 2 * (dk + dv) + 2 * T + 80, 2.0 ** -16)
    for name in ("o", "dq", "dk", "dv"):
        x = got[name]
        assert x.dtype == torch.bfloat16
        g = x.double().cpu().numpy().reshape(ref[name].shape)
        assert np.isfinite(g).all(), name
        once = torch.from_numpy(ref[name]).to(x.dtype).double().numpy()
        tol = np.abs(once - ref[name]) + 2 * E[name]
        off = np.abs(g - ref[name])
        assert (off <= tol).all(), "%s: %d of %d off, worst %.2f times the tolerance" % (
            name, (off > tol).sum(), off.size, (off / tol).max())


SHAPES = [
    # lens, H, Hkv, dk, dv, packed
    ([130, 130], 2, 1, 128, 128, False),
    ([63, 0, 65, 1, 128, 200], 3, 3, 128, 128, True),
    ([70, 129], 4, 2, 128, 64, True),
    ([100], 2, 2, 16, 96, False),
    ([77, 66], 3, 1, 57, 33, True),
    ([90, 100], 2, 2, 72, 72, True),
    ([1100, 3, 0, 3300], 2, 2, 16, 24, True),
    ([64 * 40], 1, 1, 64, 128, False),
]


@pytest.mark.parametrize("lens,H,Hkv,dk,dv,packed", SHAPES)
def test_outputs_and_gradients_are_rounded_once(lens, H, Hkv, dk, dv, packed):
    c = case("bf16", lens, H, Hkv, dk, dv, packed, seed=3)
    got = run(dev(c))
    torch.cuda.synchronize()
    check_rounded_once(c, got)


@pytest.mark.parametrize("decay", [[0.0, 0.0], [-1e-4, -0.5], [-3.0, -40.0]])
def test_rounded_once_at_any_decay(decay):
    c = case("bf16", [150, 65], 2, 2, 64, 64, True, decay=decay, seed=9)
    got = run(dev(c))
    torch.cuda.synchronize()
    check_rounded_once(c, got)


@pytest.mark.parametrize("init", [False, True])
@pytest.mark.parametrize("lens,H,Hkv,dk,dv", [([1, 2, 3, 5], 2, 1, 128, 128), ([2, 16, 2], 4, 4, 64, 40), ([2, 3], 1, 1, 33, 57)])
def test_states_are_fp32(lens, H, Hkv, dk, dv, init):
    c = case("bf16", lens, H, Hkv, dk, dv, True, init=init, seed=21)
    if not init:
        c["dS_T"] = torch.zeros_like(c["dS_T"])
    got = run(dev(c))
    torch.cuda.synchronize()
    ref, E = bounds(c, 2 * max(lens) + 16, 0.0)
    for name in ("S_T", "dS0"):
        off = np.abs(got[name].double().cpu().numpy() - ref[name])
        tol = 2.0 ** -24 * np.abs(ref[name]) + E[name]
        assert (off <= tol).all(), "%s: %d of %d off, worst %.2f times the tolerance" % (
            name, (off > tol).sum(), off.size, (off / tol).max())
