"""GPU tests of the selection of alternatives where more chunks reach the row's bound than its buffer
holds: equal maxima, as of padding rows (zero hidden states) or of repeated head rows.  The expected
ids and log-probabilities are closed forms; LP_ATOL as in test_gpu_head.py."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

LP_ATOL = 2e-5


@pytest.mark.parametrize("M", [3, 128, 200])
@pytest.mark.parametrize("V", [65536, 100008])
def test_zero_rows_over_a_long_vocabulary(lib, M, V):
    """All of a zero row's logits are equal: its alternatives are the ids 0 to k - 1.  The other rows'
    are 63 ids apart, descending."""
    W = torch.zeros((V, 16), dtype=torch.bfloat16, device="cuda")
    best = torch.arange(32, device="cuda") * 63 + 5
    W[best, 0] = (32 - torch.arange(32, device="cuda")).to(torch.bfloat16) / 4
    x = torch.zeros((M, 16), dtype=torch.bfloat16, device="cuda")
    x[1::2, 0] = 1
    zero = torch.arange(M, device="cuda") % 2 == 0
    z = W[:, 0].double()
    lse = torch.logsumexp(z, 0)
    layer = lib.LoraTokenLogProbs(lib.LoraWeight.bf16(W))
    for k in (1, 5, 32):
        for _ in range(8):
            out = layer.forward(x, None, top_k=k)
            first = torch.arange(k, dtype=torch.int32, device="cuda")
            assert torch.all(out.top_ids[zero] == first), k
            assert torch.all(out.top_ids[~zero] == best[:k].int()), k
            assert float((out.top_logprob[zero].double() + math.log(V)).abs().max()) <= LP_ATOL
            assert float((out.top_logprob[~zero].double() - (z[best[:k]] - lse)).abs().max()) <= LP_ATOL
    assert layer.status() == lib.LORA_OK
