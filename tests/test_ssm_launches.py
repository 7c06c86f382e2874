"""What the state-space layer's host code launches (no GPU: the CUDA runtime's
calls are recorded)."""
import pytest

from tests._launches import Recorder, norm_args


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
