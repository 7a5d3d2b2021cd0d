"""Pins of the oracle's token log-probabilities, entropies, alternatives and distillation:
torch's float64 functions and autograd, closed forms, finite differences."""
import numpy as np
import pytest
import torch

import oracle as O
from synth import HeadCase, make_head_case


def _case(M=9, D=24, V=40, n=3, seed=5):
    inp = make_head_case(HeadCase("t", M, D, V, n, seed))
    return inp, O.bf16_to_f64(inp["X"]), O.bf16_to_f64(inp["W"])


def _torch(X, W, T):
    x = torch.tensor(X, requires_grad=True)
    return x, torch.log_softmax(x @ torch.tensor(W).T / T, 1)


@pytest.mark.parametrize("T", [1.0, 0.7])
def test_logprobs_entropy_and_gradient_against_torch(T):
    inp, X, W = _case()
    ids = inp["ids"]
    o = O.token_logprobs(X, W, ids, -100, T, 5, inp["dlogprob"], inp["dentropy"])
    x, logp = _torch(X, W, T)
    keep = torch.tensor(ids != -100)
    lp = torch.where(keep, logp.gather(1, torch.tensor(np.where(ids >= 0, ids, 0)).long()), 0.0)
    ent = -(logp.exp() * logp).sum(1)
    assert np.allclose(o["logprob"], lp.detach().numpy(), atol=1e-12)
    assert np.allclose(o["entropy"], ent.detach().numpy(), atol=1e-12)
    val, idx = torch.topk(logp, 5, dim=1)
    assert np.allclose(o["top_logprob"], val.detach().numpy(), atol=1e-12)
    ((lp * torch.tensor(inp["dlogprob"]).double()).sum() + (ent * torch.tensor(inp["dentropy"]).double()).sum()).backward()
    assert np.allclose(o["dX"], x.grad.numpy(), atol=1e-11)


@pytest.mark.parametrize("T", [1.0, 2.5])
def test_distillation_against_torch(T):
    inp, X, W = _case(n=6)
    ids, t = inp["ids"].copy(), inp["teacher"].copy()
    ids[4] = -100          # a row without entries
    t[5] = -np.inf         # a row without mass
    t[6, 1:] = -np.inf
    o = O.distill(X, W, ids, t, -100, T, inp["dloss"])
    x, logp = _torch(X, W, T)
    keep = torch.tensor(ids != -100)
    tt = torch.where(keep, torch.tensor(t).double() / T, -torch.inf)
    q = torch.nan_to_num(torch.softmax(tt, 1), nan=0.0)
    lp = logp.gather(1, torch.tensor(np.where(ids >= 0, ids, 0)).long())
    loss = (torch.xlogy(q, q) - q * lp).sum(1)
    assert np.allclose(o["loss"], loss.detach().numpy(), atol=1e-12)
    assert o["loss"][4] == 0 and o["loss"][5] == 0 and np.all(o["dX"][[4, 5]] == 0)
    (loss * torch.tensor(inp["dloss"]).double()).sum().backward()
    assert np.allclose(o["dX"], x.grad.numpy(), atol=1e-11)


def test_closed_forms():
    X = np.zeros((2, 8))
    W = np.ones((16, 8))
    o = O.token_logprobs(X, W, [[3, 99], [-100, 3]], -100, 1.0, 4, np.ones((2, 2)), np.ones(2))
    assert np.allclose(o["logprob"], [[-np.log(16), np.nan], [0, -np.log(16)]], equal_nan=True)
    assert np.allclose(o["entropy"], np.log(16))
    assert np.array_equal(o["top_ids"], [[0, 1, 2, 3]] * 2)  # equal logits: the smaller id first
    # a uniform teacher over the whole vocabulary against a uniform student
    d = O.distill(X, W, np.tile(np.arange(16), (2, 1)), np.zeros((2, 16)), -100)
    assert np.allclose(d["loss"], 0)
    # a teacher with one entry is the cross-entropy
    inp, X, W = _case(n=1)
    d = O.distill(X, W, inp["ids"], inp["teacher"], -100, 1.0, inp["dloss"])
    loss, _, dX = O.cross_entropy(X, W, inp["ids"][:, 0], -100, inp["dloss"])
    assert np.allclose(d["loss"], loss, atol=1e-12) and np.allclose(d["dX"], dX, atol=1e-12)


def test_finite_differences():
    inp, X, W = _case(M=3, D=8, V=24, n=2)
    T, h = 1.3, 1e-6

    def f(x):
        o = O.token_logprobs(x, W, inp["ids"], -100, T)
        d = O.distill(x, W, inp["ids"], inp["teacher"], -100, T)
        return (o["logprob"] * inp["dlogprob"]).sum() + (o["entropy"] * inp["dentropy"]).sum() + \
            (d["loss"] * inp["dloss"]).sum()

    g = O.token_logprobs(X, W, inp["ids"], -100, T, 0, inp["dlogprob"], inp["dentropy"])["dX"] + \
        O.distill(X, W, inp["ids"], inp["teacher"], -100, T, inp["dloss"])["dX"]
    for m in range(3):
        for d in range(8):
            e = np.zeros_like(X)
            e[m, d] = h
            assert abs((f(X + e) - f(X - e)) / (2 * h) - g[m, d]) < 1e-6
