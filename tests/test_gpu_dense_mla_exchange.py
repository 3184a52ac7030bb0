"""Attention over the latent cache: the exchange of logits between the two halves of a pair, beside
other work that moves the pair's timing.  The caches are those whose weights are whole powers of two,
so that a logit that meets another tile's half changes a weight by a factor."""
import pytest
import torch

from indexed_sparse_attention_indexer_gb300 import binding
from tests.test_gpu_dense_mla_counts import SCALE, Marks, _spots

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H", [16, 48, 128])
def test_beside_other_work(H, fp8):
    """Long and short pieces in turn, beside copies and beside another call of the same kind: the same
    bits every time, and the formula's."""
    lens = [3000 + 257 * (i % 11) if i % 3 else 65 + i for i in range(40)]
    m = Marks(lens, len(lens), H, 64, fp8, H)
    ws = [binding.alloc_workspace(binding.dense_mla_workspace_size(len(lens), H), DEV) for _ in range(2)]
    first = binding.dense_mla_decode(m.q, m.cache, SCALE, workspace=ws[0])
    m.check(*first, [(b, b, _spots(n)) for b, n in enumerate(lens)])
    streams = [torch.cuda.Stream() for _ in range(3)]
    junk = torch.zeros((2, 1 << 26), dtype=torch.uint8, device=DEV)
    outs = [(torch.empty_like(first[0]), torch.empty_like(first[1])) for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(40):
        with torch.cuda.stream(streams[2]):
            junk[i & 1].copy_(junk[(i & 1) ^ 1])
        for s, w, (o, l) in zip(streams, ws, outs):
            o.zero_()
            s.wait_stream(torch.cuda.current_stream())
            binding.dense_mla_decode(m.q, m.cache, SCALE, out=o, lse=l, workspace=w, stream=s)
        for s, (o, l) in zip(streams, outs):
            torch.cuda.current_stream().wait_stream(s)
            assert torch.equal(o, first[0]) and torch.equal(l, first[1])
    torch.cuda.synchronize()
    assert binding.device_status() == 0
