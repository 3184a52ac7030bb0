"""Linear attention prefills at the edges of what their description promises: one short sequence in a
longer buffer, starts that go back in a call that is cut into segments."""
import math

import pytest
import torch

from indexed_sparse_attention_indexer_gb300 import binding
from tests.test_gpu_linear import DEV, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [0, 1, 5, 8])
@pytest.mark.parametrize("dk,dv", [(128, 128), (40, 24)])
def test_one_short_sequence_in_a_longer_buffer(n, dk, dv):
    """One sequence among more than 8 rows goes by chunks however short it is, with a prefill's numbers;
    without tokens it passes its state on, and rows that are not its own stay as they were."""
    c = Case([n], H=3, dk=dk, dv=dv, lead=2, tail=300, seed=n)
    c.check(*c.prefill())


@pytest.mark.parametrize("n", [1, 5, 8])
def test_short_sequences_beside_others(n):
    """Several sequences: the short ones have a step's numbers."""
    c = Case([n, 200, n], H=3, seed=n)
    out, state = c.prefill()
    c.check(out, state)
    for b, at in ((0, c.lead), (2, c.lead + n + 200)):
        ref, tol, new, tol_s = c.reference(b)
        assert bool(((out[at:at + n].double() - ref).abs() <= tol["decode"]).all())
        slot = int(c.out_slots[b])
        assert bool(((state[slot].double() - new).abs() <= tol_s["decode"]).all())
