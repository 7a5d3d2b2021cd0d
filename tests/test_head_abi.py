"""Host validation and workspace sizes of the LM head's log-probability and distillation
entries, and the layers' argument checks (no device needed)."""
import ctypes

import pytest
import torch

import qlora_linear_b200 as q
from qlora_linear_b200.binding import lora_weight_t

P, P2 = 0x10000, 0x20000  # never dereferenced: validation runs before any CUDA call
INV, ALI, UNS, WS, OK = (q.LORA_ERR_INVALID_ARG, q.LORA_ERR_ALIGNMENT, q.LORA_ERR_UNSUPPORTED, q.LORA_ERR_WORKSPACE,
                         q.LORA_OK)
M0, D0, V0 = 300, 256, 1000


def _w(fmt=0, N=V0, K=D0, data=P):
    return lora_weight_t(fmt, 0, N, K, data, P, P)


def lp_fwd(W=_w(), M=M0, X=P, ids=P, n=2, scale=1.0, k=4, lp=P, ent=P, lse=P, ti=P, tl=P, saved=None, ws=P2, nb=1 << 32):
    return q.lib().lora_logprob_fwd(X, M, ctypes.byref(W) if W is not None else None, ids, n, -100, scale, k, lp, ent,
                                    lse, ti, tl, saved, ws, nb, None)


def lp_bwd(W=_w(), M=M0, X=P, ids=P, n=2, scale=1.0, lse=P, ent=P, dlp=P, dent=P, saved=None, dX=P, ws=P2, nb=1 << 32):
    return q.lib().lora_logprob_bwd(X, M, ctypes.byref(W) if W is not None else None, ids, n, -100, scale, lse, ent,
                                    dlp, dent, saved, dX, ws, nb, None)


def kd_fwd(W=_w(), M=M0, X=P, ids=P, t=P, n=2, scale=1.0, loss=P, lse=P, saved=None, ws=P2, nb=1 << 32):
    return q.lib().lora_distill_fwd(X, M, ctypes.byref(W) if W is not None else None, ids, t, n, -100, scale, loss, lse,
                                    saved, ws, nb, None)


def kd_bwd(W=_w(), M=M0, X=P, ids=P, t=P, n=2, scale=1.0, lse=P, dl=P, saved=None, dX=P, ws=P2, nb=1 << 32):
    return q.lib().lora_distill_bwd(X, M, ctypes.byref(W) if W is not None else None, ids, t, n, -100, scale, lse, dl,
                                    saved, dX, ws, nb, None)


@pytest.mark.parametrize("call", [lp_fwd, lp_bwd, kd_fwd, kd_bwd])
def test_common_refusals(call):
    assert call(W=None) == INV
    assert call(W=_w(fmt=1, N=1000, K=256)) == UNS      # the head is bf16
    assert call(W=_w(N=1001)) == UNS and call(W=_w(K=252)) == UNS
    assert call(W=_w(data=P + 8)) == ALI
    assert call(M=-1) == INV and call(M=0, X=None, ids=None) == OK
    assert call(X=None) == INV and call(X=P + 4) == ALI
    assert call(ids=None) == INV and call(ids=P + 4) == ALI
    assert call(n=-1) == INV and call(n=129) == UNS
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=bad) == INV, bad
    assert call(lse=None) == INV and call(lse=P + 8) == ALI
    assert call(saved=P + 8) == ALI
    assert call(ws=None) == WS and call(ws=P2 + 8) == ALI and call(nb=1000) == WS


def test_forward_refusals():
    assert lp_fwd(k=-1) == INV and lp_fwd(k=33) == UNS
    assert lp_fwd(W=_w(N=8), k=9) == UNS                # more alternatives than entries
    assert lp_fwd(lp=None) == INV and lp_fwd(ent=P + 4) == ALI
    assert lp_fwd(ti=None) == INV and lp_fwd(tl=P + 4) == ALI
    need = q.head_fwd_workspace_bytes(M0, D0, V0, 2, 4)
    assert lp_fwd(nb=need // 2) == WS
    assert kd_fwd(n=0) == INV and kd_fwd(t=None) == INV and kd_fwd(t=P + 4) == ALI and kd_fwd(loss=None) == INV


def test_backward_refusals():
    assert lp_bwd(dX=None) == INV and lp_bwd(dX=P + 8) == ALI and lp_bwd(dlp=P + 4) == ALI
    assert lp_bwd(dent=P + 4) == ALI and lp_bwd(ent=None) == INV
    assert kd_bwd(n=0) == INV and kd_bwd(t=None) == INV and kd_bwd(dl=None) == INV and kd_bwd(dX=None) == INV
    # a saved forward needs no room for dz, a recomputing one room for at least 256 columns
    for call in (lp_bwd, kd_bwd):
        assert call(nb=q.head_bwd_workspace_bytes(M0, D0, V0, 2, 0) - 1, saved=P) == WS
        assert call(nb=q.head_bwd_workspace_bytes(M0, D0, V0, 2, 256) - M0 * 2) == WS


def test_workspace_sizes():
    f, b, s = q.head_fwd_workspace_bytes, q.head_bwd_workspace_bytes, q.head_saved_bytes
    assert f(300, 256, 1000, 2, 4) > f(300, 256, 1000, 2, 0) > 0
    assert f(300, 256, 1000, 129, 0) == 0 and f(300, 256, 1000, 1, 33) == 0 and f(-1, 256, 1000, 1, 1) == 0
    # rows are worked off in chunks: the scratch stops growing
    assert f(1 << 20, 4096, 128256, 1, 32) == f(1 << 16, 4096, 128256, 1, 32) <= 1281 << 20
    assert f(0, 64, 256, 0, 0) >= 256
    assert b(300, 256, 1000, 2, 256) < b(300, 256, 1000, 2, 512)
    assert b(300, 256, 1000, 2, 1000) == b(300, 256, 1000, 2, 4096)
    assert b(300, 256, 1000, 2, -1) == 0 and b(300, 0, 1000, 2, 0) == 0
    assert s(16384, 128256, 1) >= 2 * 16384 * 128256 and s(-1, 8, 1) == 0 and s(4, 0, 1) == 0 and s(4, 8, 129) == 0


def test_layer_refusals():
    W = q.LoraWeight.bf16(torch.zeros((64, 32), dtype=torch.bfloat16))
    for cls in (q.LoraTokenLogProbs, q.LoraDistill):
        with pytest.raises(ValueError):
            cls(W, temperature=0.0)
        with pytest.raises(ValueError):
            cls(W, temperature=float("nan"))
        with pytest.raises(q.LoraError):
            cls(q.LoraWeight(64, 64, P, P, P))
    with pytest.raises(ValueError):  # no CPU path
        q.LoraTokenLogProbs(W).forward(torch.zeros((2, 32), dtype=torch.bfloat16))
