"""GPU tests of what the LM head's operators keep of a result's digits."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [0, 4])
@pytest.mark.parametrize("T", [1.0, 0.01])
@pytest.mark.parametrize("M", [3, 128, 200])
def test_a_certain_token_keeps_its_digits(lib, M, T, k):
    """One entry 40/T or more above all others: its log-probability is above -1e-13 and so 0 here,
    whatever its logit's size.  Every sum of products is exact and the entry's own term is the sum: what
    remains is its 2^d (2^-22), the logarithm (2^-23) and the last rounding, below TOL = 2^-21."""
    TOL = 2.0 ** -21
    V = 1000
    W = torch.zeros((V, 16), dtype=torch.bfloat16, device="cuda")
    W[777, 0] = 8.0
    x = torch.zeros((M, 16), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 5 + (torch.arange(M, device="cuda") % 96) / 16  # logits of 40/T to 87.5/T, exact in bf16
    ids = torch.full((M, 1), 777, dtype=torch.int32, device="cuda")
    layer = lib.LoraTokenLogProbs(lib.LoraWeight.bf16(W), temperature=T)
    out = layer.forward(x, ids, top_k=k)
    assert float(out.logprob.abs().max()) <= TOL
    assert float(out.entropy.abs().max()) <= 2 * TOL
    if k:
        assert torch.all(out.top_ids[:, 0] == 777)
        assert float(out.top_logprob[:, 0].abs().max()) <= TOL
    assert layer.status() == lib.LORA_OK
