"""FP8 prefixes on both sides of what the workspace has room for (65536 positions are converted into it, by the
table's capacity), with several groups of rows, against the formula in 64 bits; tolerances of
test_gpu_prefix_mla."""
import pytest
import torch

from indexed_sparse_attention_indexer_gb300 import binding
from tests.test_gpu_prefix_mla import Shared

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prefix,capacity,page", [
    (65535, None, 0), (65536, None, 64), (65537, None, 0), (65530, 65536, 16), (65000, 65537, 0), (32768, 131072, 64),
    (131071, None, 64), (70, 65536, 64), (1, 131072, 0), (0, 65536, 64)])
def test_fp8_prefix_lengths_and_capacities(prefix, capacity, page):
    case = Shared(prefix, [5 * i % 70 for i in range(40)], 1, 16, page, True, seed=prefix % 97, prefix_max=capacity).device()
    assert case.prefix.struct.s_max >= (capacity or prefix)
    a = case.run()
    b = case.run()
    torch.cuda.synchronize()
    case.check(*a, rows=[0, 7, 8, 14, 39])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_a_workspace_that_earlier_calls_left_full():
    """Calls of other sizes and types in one workspace, one after another: each as in a workspace of its own."""
    cases = [Shared(5000, [40, 1, 300, 0] * 8, 1, 16, 64, True, seed=1), Shared(300, [9, 0, 700], 2, 64, 16, False, seed=2),
             Shared(4005, [37 * i % 200 for i in range(20)], 1, 128, 64, True, seed=3), Shared(1, [1], 1, 1, 0, False, seed=4)]
    size = max(binding.prefix_mla_workspace_size(len(c.lens) * c.T, c.H) for c in cases)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    alone = []
    for c in cases:
        c.device()
        alone.append(c.run())
    for _ in range(2):
        for c, (out, lse) in zip(cases, alone):
            y = c.run(workspace=ws)
            assert torch.equal(y[0], out) and torch.equal(y[1], lse)
    assert binding.device_status() == 0
