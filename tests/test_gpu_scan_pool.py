"""States of a serving batch's pool after a prompt and the tokens behind it, every one of them.  Tolerances as in
test_gpu_scan.py."""
import pytest
import torch

import chunk_wise_weight_amd as cw
from tests.test_gpu_scan import DTYPES, TOL_S, make, oracle, rel

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_state_of_a_prompt_and_its_tokens(dtype):
    """A prompt, then ten tokens of each row in a pool: every named state against the sequence's, the others' bits."""
    *args, D, bias = make(2, 4, 2, 200, 64, 128, dtype)
    kw = dict(D=D, dt_bias=bias, softplus=True)
    cut = lambda a, b: [v[:, :, a:b] if v.dim() > 1 else v for v in args]
    S = cw.ttt_selective_scan(*cut(0, 190), **kw)[1]
    pool = torch.randn(5, 4, 64, 128, generator=torch.Generator().manual_seed(1)).cuda()
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    pool[slots.long()] = S
    before = pool.clone()
    for t in range(190, 200):
        cw.ttt_selective_scan_step(*(v[:, :, t].contiguous() if v.dim() > 1 else v for v in args), pool, slots=slots, **kw)
    for b in range(2):
        _, Sr = oracle(b, args, D, bias, True)
        assert rel(pool[slots[b]], Sr) <= 2 * TOL_S, b
    assert torch.equal(pool[[0, 2, 4]], before[[0, 2, 4]])
