"""What the state-space layer's host code launches (no GPU: the CUDA runtime's
calls are recorded)."""
import pytest

from tests._launches import Recorder, conv_args, norm_args, scan_bwd_args
from tests.test_gpu_ssm_paths import CONV_RUNS, MANY_ITEMS, ragged


@pytest.fixture(scope="module")
def rec(tmp_path_factory):
    return Recorder(tmp_path_factory.mktemp("recorder"))


def test_shared_memory_limits_never_fall(rec):
    # Host threads may call at the same time, and a kernel's limit is the
    # device's: one thread must not lower it between another's limit and launch.
    limits, most = {}, {}
    widths = [16384, 16383, 8192, 8190, 4096, 4100, 2048, 2047, 1024, 1001, 256, 64, 7]
    for D in widths + widths[::-1]:
        for rows in (5, 700):
            for dtype in (0, 1):
                for gate in (False, True):
                    for bwd in (False, True):
                        name = "mdn_norm_residual_" + ("bwd" if bwd else "fwd")
                        for e in rec.calls(name, *norm_args(rows, D, dtype, gate, bwd)):
                            if e.limit is None:
                                most[e.kernel] = max(most.get(e.kernel, 0), e.shared)
                                # what a kernel may have without asking; its static arrays take some of it
                                assert e.shared <= limits.get(e.kernel, 47 * 1024), (D, rows, dtype, gate, bwd)
                            else:
                                assert e.limit >= limits.get(e.kernel, 0), (D, rows, dtype, gate, bwd)
                                limits[e.kernel] = e.limit
    assert len(limits) > 8 and len(most) > 20
    assert all(limit <= 227 * 1024 - 512 for limit in limits.values())


DTYPE = {"fp32": 0, "bf16": 1}


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("dtype,D,tokens", CONV_RUNS)
def test_convolution_runs_hold_many_batches(rec, dtype, D, tokens, bwd):
    # D at least 128 packets: a block is one run of 128 packets
    V = 4 if D % 4 == 0 else 2 if D % 2 == 0 and dtype == "bf16" else 1
    first = rec.calls("mdn_short_conv_" + ("bwd" if bwd else "fwd"),
                      *conv_args(len(ragged(tokens, D)), True, tokens, D, 4, DTYPE[dtype], bwd))[0]
    assert first.limit is None and first.block == 128
    runs = first.grid // -(-D // (128 * V))
    batch = 4 if dtype == "fp32" and V == 4 else 8
    # the ring has three places
    assert -(-tokens // runs) > 4 * batch


@pytest.mark.parametrize("case", MANY_ITEMS)
def test_scan_gradient_blocks_take_several_items(rec, case):
    dtype, lens, D, N, G, packed = case
    out = rec.calls("mdn_ssm_scan_bwd", *scan_bwd_args(len(lens), packed, sum(lens), D, G, N, DTYPE[dtype]))
    main = [e for e in out if e.limit is None][-2]              # the last adds up the partial sums
    channels = {16: 64, 33: 32, 128: 16}[N]
    tiles = G * -(-D // G // channels)
    assert main.grid % tiles == 0
    # at least one item a sequence, and fewer blocks for each tile
    assert main.grid // tiles < len([n for n in lens if n]) * (2 if len(set(lens)) == 1 and lens[0] > 96 else 1)
