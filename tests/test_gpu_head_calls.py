"""GPU tests of calls of the LM head's layers that come out of order, between streams and graphs, or
after other calls of the same layer: they give the results of the call alone, or are refused."""
import pytest
import torch

from synth import HeadCase, make_head_case
from tests.gpu_helpers import dev_bf16
from tests.test_gpu_head import head, up

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("save", [False, True])
def test_a_forward_of_the_other_operator_is_refused(lib, save):
    """Before anything runs, and the saved forward still serves its own backward.  (8 rows: at this
    size neither operator's buffer holds a map of rows.)"""
    inp = make_head_case(HeadCase("swap", 8, 64, 256, 2, 301))
    lp, kd = head(lib, inp, lib.LoraTokenLogProbs), head(lib, inp, lib.LoraDistill)
    x = dev_bf16(inp["X"])
    ids, t, dl, dlp = up(inp, "ids", "teacher", "dloss", "dlogprob")
    o, d = lp.forward(x, ids, save=save), kd.forward(x, ids, t, save=save)
    with pytest.raises(ValueError):
        kd.backward(x, ids, t, o, dl)
    with pytest.raises(ValueError):
        lp.backward(x, ids, d, dlp)
    assert (o.saved is not None) == save and (d.saved is not None) == save
    a, b = lp.backward(x, ids, o, dlp), kd.backward(x, ids, t, d, dl)
    assert torch.equal(a, lp.backward(x, ids, lp.forward(x, ids, save=save), dlp))
    assert torch.equal(b, kd.backward(x, ids, t, kd.forward(x, ids, t, save=save), dl))


@pytest.mark.parametrize("op", ["logprob", "distill"])
def test_forward_and_backward_in_two_graphs(lib, op):
    """A backward captured into another graph than its forward recomputes the logits, so each of its
    replays gives the gradient, however often the forward was replayed before; so does an ordinary
    backward of a captured forward.  In one graph the saved forward serves."""
    inp = make_head_case(HeadCase("two_graphs", 300, 128, 3000, 4, 311))
    x = dev_bf16(inp["X"])
    ids, t, dl, dlp, dent = up(inp, "ids", "teacher", "dloss", "dlogprob", "dentropy")
    layer = head(lib, inp, lib.LoraTokenLogProbs if op == "logprob" else lib.LoraDistill)

    def fwd(save):
        return layer.forward(x, ids, save=save) if op == "logprob" else layer.forward(x, ids, t, save=save)

    def bwd(o):
        return layer.backward(x, ids, o, dlp, dent) if op == "logprob" else layer.backward(x, ids, t, o, dl)

    saved_way, recomputed = bwd(fwd(True)), bwd(fwd(False))
    assert not torch.equal(saved_way, recomputed)
    torch.cuda.synchronize()
    a, b, both = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(a):
        o = fwd(True)
    with torch.cuda.graph(b):
        got = bwd(o)
    with torch.cuda.graph(both):
        together = bwd(fwd(True))
    for replays in (1, 3, 2):
        a.replay()
        for _ in range(replays):
            got.zero_()
            b.replay()
            torch.cuda.synchronize()
            assert torch.equal(got, recomputed)
        assert torch.equal(bwd(o), recomputed) and torch.equal(bwd(o), recomputed)
        together.zero_()
        both.replay()
        torch.cuda.synchronize()
        assert torch.equal(together, saved_way)
    del a, b, both


@pytest.mark.parametrize("op", ["logprob", "distill"])
def test_slices_are_those_of_the_call_whatever_ran_before(lib, op):
    """The slices of a backward that recomputes go by the layer's slice_, not by what a larger call
    left as its workspace: the same bits before and after one, and in a graph."""
    inp = make_head_case(HeadCase("grown", 300, 128, 5000, 4, 321))
    x = dev_bf16(inp["X"])
    ids, t, dl, dlp, dent = up(inp, "ids", "teacher", "dloss", "dlogprob", "dentropy")
    W = lib.LoraWeight.bf16(dev_bf16(inp["W"]))
    cls = lib.LoraTokenLogProbs if op == "logprob" else lib.LoraDistill

    def bwd(layer, o):
        return layer.backward(x, ids, o, dlp, dent) if op == "logprob" else layer.backward(x, ids, t, o, dl)

    whole = cls(W)
    o = whole.forward(x, ids) if op == "logprob" else whole.forward(x, ids, t)
    one_piece = bwd(whole, o)
    layer = cls(W, slice_=256)
    want = bwd(layer, o)
    assert not torch.equal(want, one_piece)
    before = sum(ws.numel() for ws in layer._ws.values())
    big = x.repeat(8, 1)
    if op == "logprob":
        layer.forward(big, None, top_k=32)
    else:
        layer.forward(big, ids.repeat(8, 1), t.repeat(8, 1))
    assert sum(ws.numel() for ws in layer._ws.values()) > before
    assert torch.equal(bwd(layer, o), want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = bwd(layer, o)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    del g


def test_a_refused_backward_keeps_the_saved_forward(lib):
    """Other sizes than the forward's, a tensor that does not start on 16 bytes: the call is refused and
    the saved forward still serves the right one."""
    inp = make_head_case(HeadCase("refused", 300, 64, 1000, 2, 331))
    x = dev_bf16(inp["X"])
    ids, dlp = up(inp, "ids", "dlogprob")
    layer = head(lib, inp, lib.LoraTokenLogProbs)
    want = layer.backward(x, ids, layer.forward(x, ids, save=True), dlp)
    o = layer.forward(x, ids, save=True)
    with pytest.raises(ValueError):
        layer.backward(x, ids[:, 0].contiguous(), o, dlp[:, 0].contiguous())
    assert o.saved is not None
    off = torch.empty(601, dtype=torch.int32, device="cuda")[1:].view(300, 2)
    off.copy_(ids)
    with pytest.raises(lib.LoraError):
        layer.backward(x, off, o, dlp)
    assert o.saved is not None
    assert torch.equal(layer.backward(x, ids, o, dlp), want) and o.saved is None


@pytest.mark.parametrize("what", ["dX", "head"])
def test_tensors_of_another_stream_are_kept_until_the_call_has_run(lib, what):
    """A caller's dX and the head, dropped by the caller right after a call on another stream: their
    memory is not handed out before that call has run."""
    inp = make_head_case(HeadCase("drop", 300, 136, 3000, 4, 341))
    x = dev_bf16(inp["X"])
    ids, t, dl = up(inp, "ids", "teacher", "dloss")
    layer = head(lib, inp, lib.LoraDistill)
    s = torch.cuda.Stream()
    o = layer.forward(x, ids, t)
    torch.cuda.synchronize()
    # a workspace of the stream, so that the call itself takes nothing large from the allocator
    want = layer.backward(x, ids, t, o, dl, stream=s)
    torch.cuda.synchronize()
    dX = torch.empty_like(x)
    torch.cuda.synchronize()
    kept = dX if what == "dX" else layer.W.data
    where, shape = kept.data_ptr(), kept.shape
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)  # about 0.1 s, before the backward in its stream
    got = layer.backward(x, ids, t, o, dl, dX=dX, stream=s)
    assert got is dX
    del kept, got
    if what == "dX":
        del dX
    else:
        del layer
    other = [torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    assert all(a.data_ptr() != where for a in other)
    torch.cuda.synchronize()
    if what == "head":
        assert torch.equal(dX, want)


def test_a_wrong_dX_is_refused_on_every_stream(lib):
    inp = make_head_case(HeadCase("wrong_dX", 8, 64, 256, 2, 351))
    lp, kd = head(lib, inp, lib.LoraTokenLogProbs), head(lib, inp, lib.LoraDistill)
    x = dev_bf16(inp["X"])
    ids, t, dl, dlp = up(inp, "ids", "teacher", "dloss", "dlogprob")
    o, d = lp.forward(x, ids), kd.forward(x, ids, t)
    torch.cuda.synchronize()
    for stream in (None, torch.cuda.Stream()):
        for dX in (torch.empty_like(x, device="cpu"), torch.empty_like(x)[:4], x.float(), "dX"):
            with pytest.raises(ValueError):
                lp.backward(x, ids, o, dlp, dX=dX, stream=stream)
            with pytest.raises(ValueError):
                kd.backward(x, ids, t, d, dl, dX=dX, stream=stream)
