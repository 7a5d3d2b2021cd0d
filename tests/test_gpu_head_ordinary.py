"""GPU tests of the LM head's operators on ordinary bf16 normals, whose sums of products are not exact
in fp32 (the other tests' grids make them so), against plain formulas in 64 bits.

Tolerances.  A logit is summed in D/16 steps of 16 products.  Published measurements of tensor cores
(Fasi, Higham, Mikaitis, Pranesh, 2021) find a step's addends aligned to the largest and cut off at two
or more bits below fp32: at most 17·2^-25 < 2^-20 of the largest magnitude a step.  That magnitude is
at most a partial sum, which, as the few-row kernel starts at any column, is at most 3·max|S_k| over
the sums S_k of the first k steps, or one step's Σ|x·w|.  So a logit is off by
e = (D/16)·2^-20·(3·max|S_k| + max Σ_step |x·w|), and by its scaling.  Log-probabilities and losses are
off by twice that (logit and normaliser) on top of the bounds of test_gpu_head.py; the entropy, whose
derivative in z_v is -p_v·(log p_v + H), by e·Σp|log p + H| <= 2·H·e; p, and with it dz, by 2·e
relative: 2·e·scale·Σ|c|·(p·|W|) in dX."""
import pytest
import torch

from tests.test_gpu_head import ENT_ATOL, LOSS_ATOL, LP_ATOL

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,D,V,T", [(48, 4096, 2056, 1.0), (48, 8192, 1000, 0.7), (300, 4096, 1000, 1.0),
                                     (300, 8192, 2056, 1.0)])
def test_ordinary_values(lib, M, D, V, T):
    g = torch.Generator(device="cuda").manual_seed(M + D + V)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    W = (normal(V, D) * (2.0 / D ** 0.5)).to(torch.bfloat16)
    x = normal(M, D).to(torch.bfloat16)
    n, k = 3, 6
    ids = torch.randint(0, V, (M, n), generator=g, device="cuda", dtype=torch.int32)
    dlp, t, dl = normal(M, n), 2 * normal(M, n), normal(M).abs() + 0.5
    Xd, Wd = x.double(), W.double()
    steps = torch.bmm(Xd.view(M, -1, 16).transpose(0, 1), Wd.view(V, -1, 16).permute(1, 2, 0))
    size = torch.bmm(Xd.abs().view(M, -1, 16).transpose(0, 1), Wd.abs().view(V, -1, 16).permute(1, 2, 0))
    e = float(D / 16 * 2.0 ** -20 / T * (3 * steps.cumsum(0).abs().max() + size.max()))
    del steps, size
    z = Xd @ Wd.T / T
    logp = torch.log_softmax(z, 1)
    p = logp.exp()
    H = -(p * logp).sum(1)
    idl = ids.long()
    lp = logp.gather(1, idl)
    q = torch.softmax(t.double() / T, 1)
    loss = (q * (q.log() - lp)).sum(1)
    worst = {}

    def near(name, got, ref, tol):
        worst[name] = float((got.double() - ref).abs().max())
        assert worst[name] <= tol, (name, worst[name], tol)

    def near_dX(name, got, c):
        dz = (-p * c.sum(1, keepdim=True)).scatter_add(1, idl, c) / T
        ref = dz @ Wd
        total = c.abs().sum(1, keepdim=True)
        bound = (2 * 2.0 ** -8 + 2.0 ** -10) * (dz.abs() @ Wd.abs()) + 2.0 ** -8 * ref.abs() + \
            (2.0 ** -8 + 2 * e) / T * total * (p @ Wd.abs())
        worst[name] = float(((got.double() - ref).abs() / bound).max())
        assert worst[name] <= 1, (name, worst[name])

    head = lib.LoraWeight.bf16(W)
    a, b = lib.LoraTokenLogProbs(head, temperature=T), lib.LoraDistill(head, temperature=T)
    for save in (False, True):
        o, d = a.forward(x, ids, top_k=k, save=save), b.forward(x, ids, t, save=save)
        near("logprob", o.logprob, lp, 2 * e + LP_ATOL)
        near("entropy", o.entropy, H, 2 * float(H.max()) * e + ENT_ATOL)
        near("top", o.top_logprob, logp.topk(k, 1)[0], 2 * e + LP_ATOL)
        near("top ids", o.top_logprob, logp.gather(1, o.top_ids.long()), 2 * e + LP_ATOL)
        near("loss", d.loss, loss, 2 * e + LOSS_ATOL)
        near_dX("dX", a.backward(x, ids, o, dlp), dlp.double())
        near_dX("distill dX", b.backward(x, ids, t, d, dl), -dl.double()[:, None] * q)
    print(f"e = {e:.1e}", {name: f"{v:.1e}" for name, v in worst.items()})
    assert a.status() == lib.LORA_OK and b.status() == lib.LORA_OK
