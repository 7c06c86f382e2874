"""The group norm on the GPU: calls and paths beside those of
test_gpu_group_norm.py (its tolerances)."""
import pytest
import torch

from tests.test_gpu_group_norm import case, check_case, dev, run

pytestmark = pytest.mark.gpu

MANY = [
    # more sequences than the gradient has clusters: packed ones that fit shared memory, and equal ones
    ([i % 3 for i in range(300)], 2048, 16, True),
    ([2] * 1000, 48, 3, False),
    # ... and than it has blocks for tiles, where the batch is too long for shared memory
    ([(7 * i) % 4 for i in range(4000)], 512, 1, True),
    ([0, 5000] + [1] * 700, 64, 4, True),
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("lens,D,G,packed", MANY)
def test_more_sequences_than_sums(dtype, gate, lens, D, G, packed):
    check_case(case(dtype, lens, D, G, gate, over="sequence", packed=packed, seed=len(lens)))


@pytest.mark.parametrize("lens,D,G,packed", MANY)
def test_their_workspace_holds_what_is_written(lens, D, G, packed):
    import momentum_delta_rule_gb300 as mdn
    d = dev(case("bf16", lens, D, G, over="sequence", packed=packed))
    want = run(d)
    need = mdn.lib().mdn_group_norm_bwd_workspace_size(len(lens), sum(lens), D, G, 1, mdn.MDN_BF16)
    ws = torch.full((need + 4096,), 0x55, dtype=torch.uint8, device="cuda")
    g = mdn.group_norm_bwd(d["x"], G, want["stats"], d["dy"], weight=d["weight"], bias=d["bias"], gate=d["gate"], activation="silu",
                           over="sequence", cu_seqlens=d["cu"], workspace=ws[:need])
    assert all(torch.equal(g[n], want[n]) for n in g)
    assert (ws[need:] == 0x55).all()
