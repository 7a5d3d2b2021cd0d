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


@pytest.mark.parametrize("M", [3, 128, 200])
@pytest.mark.parametrize("V,step", [(200000, 160), (262144, 160), (151936, 144), (200000, 32), (300008, 4000)])
def test_repeated_best_entries_past_4608_chunks(lib, M, V, step):
    """More chunks than the selection looks at in one pass (4608), with fewer than its buffer's 1024
    tied for the best in the first pass and more with the next ones (151936 by 144: 1024 and 32), or
    one in every chunk.  Odd rows have all other entries tied for the best."""
    W = torch.zeros((V, 16), dtype=torch.bfloat16, device="cuda")
    W[::step, 0] = 1.0
    x = torch.zeros((M, 16), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1
    x[1::2, 0] = -1
    odd = torch.arange(M, device="cuda") % 2 == 1
    peaks = -(-V // step)
    lse_even = math.log(peaks * math.e + (V - peaks))
    lse_odd = math.log(peaks / math.e + (V - peaks))
    others = torch.tensor([v for v in range(100) if v % step][:32], dtype=torch.int32, device="cuda")
    layer = lib.LoraTokenLogProbs(lib.LoraWeight.bf16(W))
    for k in (1, 2, 5, 32):
        out = layer.forward(x, None, top_k=k)
        assert torch.all(out.top_ids[~odd] == torch.arange(k, dtype=torch.int32, device="cuda") * step), k
        assert torch.all(out.top_ids[odd] == others[:k]), k
        assert float((out.top_logprob[~odd].double() - (1 - lse_even)).abs().max()) <= LP_ATOL
        assert float((out.top_logprob[odd].double() + lse_odd).abs().max()) <= LP_ATOL
    assert layer.status() == lib.LORA_OK
