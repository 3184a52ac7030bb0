"""Linear attention prefills at the edges of what their description promises: one short sequence in a
longer buffer, starts that go back in a call that is cut into segments."""
import pytest
import torch

from indexed_sparse_attention_indexer_gb300 import binding
from tests.test_gpu_linear import DEV, Case
from tests.test_gpu_linear_split import Prompts

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


@pytest.mark.parametrize("H,B", [(1, 3), (2, 5), (1, 9)])
def test_starts_that_go_back_over_a_cut_prompt(H, B):
    """Every other sequence has all the tokens, which is more segments than the workspace is meant for: the
    call reports it, writes nothing beyond the workspace, and every sequence has its outputs and its state,
    those of a call that leaves it whole."""
    n, d = 30000, 64
    p = Prompts([n], H, d)
    p.call(False)
    size = binding.linear_workspace_size(n, B, H, d, d)
    assert size > 256
    ws = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
    starts = torch.tensor([b % 2 * n for b in range(B + 1)], dtype=torch.int32, device=DEV)
    state = torch.full((B, H, d, d), 3.0, device=DEV)
    slots = torch.arange(B, dtype=torch.int32, device=DEV)
    out = binding.linear_prefill(p.q, p.k, p.v, p.decay, d ** -0.5, starts, state, torch.full_like(slots, -1), slots,
                                 workspace=ws[:size])
    assert binding.device_status() == binding.DSI_ERR_BOUNDS
    assert bool((ws[size:] == 0x5A).all())
    assert torch.equal(out, p.out)
    for b in range(B):
        assert torch.equal(state[b], p.state[0] if b % 2 == 0 else torch.zeros_like(state[b])), b


@pytest.mark.parametrize("lens,H", [([5000] + [1] * 3, 2), ([1] * 20 + [5000] + [3] * 20, 2), ([40] * 7 + [6000], 1),
                                    ([2, 3000] * 4, 4), ([1] * 63 + [4000], 1), ([1] * 64 + [4000], 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_a_long_prompt_beside_short_rows(lens, H, d):
    """Cut, or left whole for its neighbours' sake: against the formula either way."""
    c = Case(lens, H=H, dk=d, dv=d, seed=len(lens))
    c.check(*c.prefill())


@pytest.mark.parametrize("where", ["q", "k", "v"])
@pytest.mark.parametrize("at", [0, 100, 200])
def test_what_a_bad_value_does_not_reach_follows_the_formula(where, at):
    """Tokens before it, other heads and the next sequence, in outputs and states."""
    c = Case([260, 90], H=3, lead=0, tail=0, seed=31)
    {"q": c.dq, "k": c.dk_, "v": c.dv_}[where][at, 1, 7] = float("nan")
    out, state = c.prefill()
    assert binding.device_status() == 0
    for b, (lo, hi) in enumerate(((0, 260), (260, 350))):
        ref, tol, new, tol_s = c.reference(b)
        ok = torch.ones(ref.shape, dtype=torch.bool, device=DEV)
        heads = [0, 1, 2]
        if b == 0:
            ok[at:at + 1 if where == "q" else 260, 1] = False
            heads = [0, 1, 2] if where == "q" else [0, 2]
        assert bool((((out[lo:hi].double() - ref).abs() <= tol["prefill"]) | ~ok).all())
        slot = int(c.out_slots[b])
        assert bool(((state[slot].double() - new).abs() <= tol_s["prefill"])[heads].all())
