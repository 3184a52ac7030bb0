"""The state that a prefill of linear attention leaves, value by value, where no sum hides what one token
adds: keys with one dim each, 2^e, so that row j of the state is 2^e exp(g (n - 1 - j)) v_j.

Tolerance: the exponential is off by two units (2 * 2^-23 of it) and its angle, of at most 4, by half a
step (4 * 2^-24); the product with v rounds once (2^-24); the tensor core adds three parts, each of which it may
cut off (3 * 2^-23).  Together 15 * 2^-24 < 2^-20 of the value.
"""
import pytest
import torch

from indexed_sparse_attention_indexer_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("lens", [[128], [100, 128, 9, 77], [64] * 300])
@pytest.mark.parametrize("dv", [128, 64, 24])
def test_what_a_token_adds_keeps_its_bits(lens, dv):
    H, dk = 4, 128
    g = torch.Generator(device=DEV).manual_seed(len(lens) + dv)
    starts = torch.tensor([0] + lens, device=DEV).cumsum(0)
    n = sum(lens)
    j = torch.arange(n, device=DEV) - starts[:-1].repeat_interleave(torch.tensor(lens, device=DEV))
    size = torch.exp2(torch.randint(-3, 4, (n, H), generator=g, device=DEV).float())
    k = torch.zeros((n, H, dk), device=DEV).scatter_(2, j[:, None, None].expand(n, H, 1), size[..., None]).to(torch.bfloat16)
    q = torch.randn((n, H, dk), generator=g, device=DEV).to(torch.bfloat16)
    v = torch.randn((n, H, dv), generator=g, device=DEV).to(torch.bfloat16)
    decay = torch.tensor([-0.031, -0.0173, -0.0071, -0.0009], device=DEV)
    state = torch.zeros((len(lens), H, dk, dv), device=DEV)
    binding.linear_prefill(q, k, v, decay, 1.0, starts.to(torch.int32), state)
    assert binding.device_status() == 0
    for b, m in enumerate(lens):
        rows = slice(int(starts[b]), int(starts[b]) + m)
        left = torch.exp(decay.double()[:, None] * (m - 1 - torch.arange(m, device=DEV)))             # [H, m]
        want = (left * size[rows].double().t())[..., None] * v[rows].double().transpose(0, 1)
        assert bool(((state[b, :, :m].double() - want).abs() <= 2.0 ** -20 * want.abs()).all()), b
        assert not bool(state[b, :, m:].any())
